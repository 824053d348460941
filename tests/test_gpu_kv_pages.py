"""Reserving, forking, freeing, compacting and copying pages on the GPU against a plain model of the tables."""
import numpy as np
import pytest
import torch

from attn_helpers import DEV, i32

pytestmark = pytest.mark.gpu

BAD, NONE_LEFT = 3, 4


class Model:
    def __init__(self, rows, max_pages, num_pages, page):
        self.table, self.refs = np.zeros((rows, max_pages), np.int32), np.zeros(num_pages, np.int32)
        self.len, self.page = np.zeros(rows, np.int32), page

    def free_pages(self):
        return [p for p in range(1, len(self.refs)) if self.refs[p] == 0]

    def held(self, r):
        return int((self.table[r] != 0).sum())

    def reserve(self, rows, tokens):
        free, status, asked = self.free_pages(), [], 0
        for r, n in zip(rows, tokens):
            if not (0 <= r < len(self.len) and 0 <= n <= self.table.shape[1] * self.page):
                status.append(BAD)
                continue
            have = self.held(r)
            ask = max(0, -(-n // self.page) - have)
            if asked + ask > len(free) and ask:
                status.append(NONE_LEFT)
            else:
                for j in range(ask):
                    self.table[r, have + j] = free[asked + j]
                    self.refs[free[asked + j]] = 1
                status.append(0)
            asked += ask
        return status

    def fork(self, src, dst):
        free, status, moves, asked = self.free_pages(), [], [], 0
        plan = []
        for s, d in zip(src, dst):
            if not (0 <= s < len(self.len) and 0 <= d < len(self.len) and s != d) or self.table[d, 0] != 0:
                status.append(BAD)
                continue
            n = int(self.len[s])
            full, part = n // self.page, n % self.page > 0
            if part:
                asked += 1
                if asked > len(free):
                    status.append(NONE_LEFT)
                    continue
                moves.append((int(self.table[s, full]), free[asked - 1]))
            plan.append((s, d, full, free[asked - 1] if part else 0))
            status.append(0)
        for s, d, full, page in plan:
            self.table[d] = 0
            self.table[d, :full] = self.table[s, :full]
            np.add.at(self.refs, self.table[d, :full], 1)
            if page:
                self.table[d, full] = page
                self.refs[page] = 1
            self.len[d] = self.len[s]
        return status, moves

    def free(self, rows):
        for r in rows:
            for p in self.table[r]:
                if p:
                    self.refs[p] -= 1
            self.table[r] = 0
            self.len[r] = 0

    def compact(self):
        live = self.refs > 0
        live[0] = True
        n = int(live.sum())
        at = np.arange(len(live))
        src, dst = at[live & (at >= n)], at[~live & (at < n)]
        remap = np.where(live, at, 0)
        remap[src] = dst
        refs = self.refs.copy()
        refs[dst], refs[src] = refs[src], 0
        return remap, refs, remap[self.table], src, dst


class Device:
    def __init__(self, m):
        self.table, self.refs, self.len = i32(m.table), i32(m.refs), i32(m.len)

    def same(self, m):
        assert np.array_equal(self.table.cpu().numpy(), m.table)
        assert np.array_equal(self.refs.cpu().numpy()[1:], m.refs[1:])
        assert np.array_equal(self.len.cpu().numpy(), m.len)


@pytest.mark.parametrize("rows,max_pages,num_pages,page", [(9, 7, 40, 16), (60, 300, 5000, 16), (300, 9, 1300, 128)])
def test_random_lives_of_rows(gdn, rows, max_pages, num_pages, page):
    rng = np.random.default_rng(rows)
    m = Model(rows, max_pages, num_pages, page)
    d = Device(m)
    for step in range(30):
        empty = [r for r in range(rows) if m.held(r) == 0]
        full = [r for r in range(rows) if m.held(r)]
        rng.shuffle(empty)
        rng.shuffle(full)
        kind = step % 3
        if kind == 0 or not full:
            pick = (empty[: 1 + len(empty) // 3] + full[: len(full) // 4])
            rng.shuffle(pick)
            tokens = [int(rng.integers(0, max_pages * page + 1) if rng.random() < 0.5 else rng.integers(0, 3 * page)) for _ in pick]
            want = m.reserve(pick, tokens)
            got = gdn.kv_pages_reserve(d.table, d.refs, i32(pick), i32(tokens), page)
            assert got.cpu().tolist() == want
            for r, n, st in zip(pick, tokens, want):
                if st == 0:
                    m.len[r] = max(m.len[r], n)
            d.len.copy_(i32(m.len))
        elif kind == 1 and empty:
            dst = empty[: 1 + len(empty) // 2]
            src = [full[i] for i in rng.integers(0, len(full), len(dst))]
            status, moves = m.fork(src, dst)
            mv = gdn.KVPageMoves(len(dst))
            mv.src.fill_(9), mv.dst.fill_(9)
            gdn.kv_pages_fork(d.table, d.len, d.refs, i32(src), i32(dst), page, mv)
            assert mv.status.cpu().tolist() == status
            n = int(mv.count)
            assert list(zip(mv.src.tolist(), mv.dst.tolist()))[:n] == moves
            assert not mv.src[n:].any() and not mv.dst[n:].any()
        else:
            pick = full[: 1 + len(full) // 3]
            m.free(pick)
            gdn.kv_pages_free(d.table, d.len, d.refs, i32(pick))
        d.same(m)
    assert gdn.get_device_error() in (0, NONE_LEFT)
    m.free(range(rows))
    gdn.kv_pages_free(d.table, d.len, d.refs, i32(np.arange(rows)))
    d.same(m)
    assert not m.refs.any()


def test_reservation_of_many_rows_out_of_pages(gdn):
    m = Model(4096, 4, 6000, 16)
    d = Device(m)
    tokens = np.random.default_rng(0).integers(0, 65, 4096)
    rows = np.random.default_rng(1).permutation(4096)
    want = m.reserve(rows, tokens)
    assert NONE_LEFT in want
    assert gdn.kv_pages_reserve(d.table, d.refs, i32(rows), i32(tokens), 16).cpu().tolist() == want
    d.same(m)
    assert gdn.get_device_error() == NONE_LEFT


@pytest.mark.parametrize("num_pages,live", [(1, 0), (2, 0.5), (37, 0.0), (37, 1.0), (1024, 0.5), (1025, 0.4), (4096, 0.3), (4097, 0.7), (30000, 0.5), (30000, 0.01)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compaction(gdn, num_pages, live, in_place):
    rng = np.random.default_rng(num_pages)
    m = Model(50, max(1, num_pages // 25), num_pages, 16)
    pages = 1 + rng.permutation(max(0, num_pages - 1))[: int(live * (num_pages - 1))]
    m.table.ravel()[: len(pages)] = pages
    m.table[7, : m.table.shape[1] // 2] = m.table[6, : m.table.shape[1] // 2]
    m.refs = np.bincount(m.table.ravel(), minlength=num_pages).astype(np.int32)
    d = Device(m)
    remap, refs, table, src, dst = m.compact()
    mv = gdn.KVPageMoves(num_pages)
    out = {} if in_place else dict(table_out=torch.full_like(d.table, -5), refs_out=torch.full_like(d.refs, -5))
    got = gdn.kv_pages_compact(d.table, d.refs, mv, **out)
    assert np.array_equal(got.cpu().numpy(), remap)
    assert np.array_equal((out["table_out"] if out else d.table).cpu().numpy(), table)
    assert np.array_equal((out["refs_out"] if out else d.refs).cpu().numpy()[1:], refs[1:])
    n = int(mv.count)
    assert n == len(src) and np.array_equal(mv.src.cpu().numpy()[:n], src) and np.array_equal(mv.dst.cpu().numpy()[:n], dst)
    assert not mv.src[n:].any() and not mv.dst[n:].any()
    if not in_place:
        d.same(m)
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,hkv,d,layers", [(16, 1, 64, 1), (16, 3, 64, 2), (128, 2, 256, 1), (32, 4, 128, 3)])
def test_copies(gdn, dtype, page, hkv, d, layers):
    pool = gdn.KVPagePool(30, page, hkv, d, layers=layers, dtype=dtype)
    pool.k.copy_(torch.randn(pool.k.shape)), pool.v.copy_(torch.randn(pool.v.shape))
    k, v = pool.k.clone(), pool.v.clone()
    mv = gdn.KVPageMoves(6)
    mv.src.copy_(i32([3, 3, 29, 0, 7, 8])), mv.dst.copy_(i32([4, 5, 1, 0, 11, 12])), mv.count.fill_(5)
    gdn.kv_pages_copy(pool, mv)
    for s, t in ((3, 4), (3, 5), (29, 1), (7, 11)):
        k[:, t], v[:, t] = k[:, s], v[:, s]
    assert torch.equal(pool.k, k) and torch.equal(pool.v, v)
    assert gdn.get_device_error() == 0
    mv.src.copy_(i32([30, 3, 3, -1, 0, 3])), mv.dst.copy_(i32([4, 0, 30, 5, 6, 2])), mv.count.fill_(100)
    gdn.kv_pages_copy(pool, mv)
    k[:, 2], v[:, 2] = k[:, 3], v[:, 3]
    assert torch.equal(pool.k, k) and torch.equal(pool.v, v)
    assert gdn.get_device_error() == BAD


def test_bad_entries_are_refused_one_by_one(gdn):
    m = Model(6, 4, 12, 16)
    d = Device(m)
    assert gdn.kv_pages_reserve(d.table, d.refs, i32([0, 6, -1, 1, 2]), i32([40, 1, 1, 65, -1]), 16).tolist() == [0, BAD, BAD, BAD, BAD]
    assert gdn.get_device_error() == BAD
    m.reserve([0], [40])
    d.same(m)
    m.len[0] = 40
    d.len[0] = 40
    mv = gdn.KVPageMoves(5)
    gdn.kv_pages_fork(d.table, d.len, d.refs, i32([0, 0, 7, 0, 0]), i32([1, 0, 2, -1, 6]), 16, mv)
    assert mv.status.tolist() == [0, BAD, BAD, BAD, BAD]
    m.fork([0], [1])
    d.same(m)
    gdn.kv_pages_fork(d.table, d.len, d.refs, i32([0, 0, 1, 0, 0]), i32([1, 2, 3, 4, 5]), 16, mv)  # 1 is taken
    assert mv.status.tolist() == [BAD, 0, 0, 0, 0]
    m.fork([0, 1, 0, 0], [2, 3, 4, 5])
    d.same(m)
    assert gdn.get_device_error() == BAD
    gdn.kv_pages_free(d.table, d.len, d.refs, i32([9, 2, 2, -3]))
    m.free([2])
    d.same(m)
    assert gdn.get_device_error() == BAD
    d.table[3, 1] = 99
    rem = gdn.kv_pages_compact(d.table, d.refs, gdn.KVPageMoves(12))
    assert gdn.get_device_error() == BAD and d.table[3, 1] == 0 and rem.shape == (12,)


def test_wrong_arguments_are_refused(gdn):
    t, refs, n = i32(np.zeros((4, 3))), i32(np.zeros(9)), i32(np.zeros(4))
    mv = gdn.KVPageMoves(1)
    with pytest.raises(gdn.GDNError):
        gdn.kv_pages_reserve(t, refs, i32([0]), i32([1]), 24)
    with pytest.raises(ValueError):
        gdn.kv_pages_reserve(t, refs, i32([0]), i32([1, 2]), 16)
    with pytest.raises(ValueError):
        gdn.kv_pages_fork(t, n, refs, i32([0, 1]), i32([2, 3]), 16, mv)
    with pytest.raises(ValueError):
        gdn.kv_pages_free(t, n[:3], refs, i32([0]))
    with pytest.raises(ValueError):
        gdn.kv_pages_compact(t, refs, mv)
    with pytest.raises(TypeError):
        gdn.kv_pages_free(t.long(), n, refs, i32([0]))
    with pytest.raises(ValueError):
        gdn.kv_pages_free(t[:, :2], n, refs, i32([0]))
    gdn.kv_pages_free(t, n, refs, i32([]))
    assert gdn.get_device_error() == 0
