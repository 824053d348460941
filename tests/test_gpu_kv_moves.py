"""KVPageMoves with room for more forks than a call makes: a loop that forks now more, now fewer rows keeps one."""
import pytest

from attn_helpers import i32
from test_gpu_kv_pages import Device, Model

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["cpp", "ctypes"])
def way(request, gdn, monkeypatch):
    from gated_deltanet_decode_gb300 import _lib
    if request.param == "ctypes":
        monkeypatch.setattr(_lib, "_fast", None)
    elif _lib.fast() is None:
        pytest.skip("the C++ binding was not built")
    return gdn


def test_lists_longer_than_the_forks(way):
    m = Model(12, 6, 60, 16)
    assert m.reserve([0, 1], [40, 70]) == [0, 0]
    m.len[:2] = 40, 70
    d, mv = Device(m), way.KVPageMoves(7)
    pool = way.KVPagePool(60, 16, 1, 64)
    pool.k.copy_(pool.k.new_tensor(range(60)).view(1, 60, 1, 1, 1).expand_as(pool.k))
    k = pool.k.clone()
    for src, dst in (([0, 1, 1, 0, 0], [2, 3, 4, 5, 6]), ([1], [7]), ([0, 1], [8, 9])):
        status, moves = m.fork(src, dst)
        assert way.kv_pages_fork(d.table, d.len, d.refs, i32(src), i32(dst), 16, mv) is mv
        n = int(mv.count)
        assert mv.status[: len(src)].tolist() == status and list(zip(mv.src.tolist(), mv.dst.tolist()))[:n] == moves
        d.same(m)
        way.kv_pages_copy(pool, mv)
        for a, b in moves:
            k[:, b] = k[:, a]
        assert (pool.k == k).all()
    assert way.get_device_error() == 0


def test_lists_shorter_than_the_forks_are_refused(way):
    m = Model(12, 6, 60, 16)
    d, mv = Device(m), way.KVPageMoves(2)
    with pytest.raises(ValueError):
        way.kv_pages_fork(d.table, d.len, d.refs, i32([0, 0, 0]), i32([1, 2, 3]), 16, mv)
    with pytest.raises(ValueError):
        way.kv_pages_compact(d.table, d.refs, mv)
    d.same(m)
