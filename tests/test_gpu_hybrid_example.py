"""The example's hybrid decoder: forks go on as their parents do, chunks give what single tokens give, and compaction
changes nothing that is computed."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("hybrid_step", os.path.join(ROOT, "examples", "hybrid_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def tokens(ex, n, seed):
    return torch.randn((n, ex.HIDDEN), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def test_it_runs(gdn, ex, capsys):
    assert ex.main()
    assert "error word 0" in capsys.readouterr().out


def test_chunks_and_single_tokens_agree(gdn, ex):
    """bf16 activations of order one through eight layers: the two ways round differently in the products, 2^-8 a layer at
    most, against 2^-8 x 8 layers x 4 for the norm of the difference."""
    x = tokens(ex, 45, 3)
    a, b = ex.Decoder(2, 64, 20), ex.Decoder(2, 64, 20)
    one = a.step(x, [40, 5])
    parts = [b.step(x[:33], [33, 0]), b.step(torch.cat([x[33:40], x[40:44]]), [7, 4]), b.step(x[44:], [0, 1])]
    two = torch.cat([parts[0], parts[1][:7], parts[1][7:], parts[2]])
    rel = (one.float() - two.float()).norm() / one.float().norm()
    assert rel < 32 * 2.0 ** -8
    assert torch.equal(a.length, b.length) and gdn.get_device_error() == 0


def test_forks_and_compaction_change_no_row(gdn, ex):
    a, b = ex.Decoder(5, 128, 60), ex.Decoder(5, 128, 60)
    x = tokens(ex, 90, 4)
    for m in (a, b):
        m.step(x, [50, 20, 20, 0, 0])
        assert m.fork([0, 2], [3, 4]).tolist() == [0, 0]
        m.release([1])
    a.compact()
    assert int(a.table.max()) < int(b.table.max()) and int(a.table.max()) == int((a.refs > 0).sum())
    for t in range(20):
        y = tokens(ex, 2, 10 + t)
        y = torch.cat([y, y])  # rows 0, 2 and their forks 3, 4
        ya, yb = (m.step(y, [1, 0, 1, 1, 1]) for m in (a, b))
        assert torch.equal(ya, yb)
        assert torch.equal(ya[0], ya[2]) and torch.equal(ya[1], ya[3])
    assert gdn.get_device_error() == 0
