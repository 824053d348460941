"""Linear attention over long sequences with decays slow enough that what a segment carries to the next one counts, and the
precision of the outputs by their norm."""
import pytest
import torch

from linear_helpers import DEV, Case, SlowCase, i32
from test_gpu_linear_attention import prefill

pytestmark = pytest.mark.gpu

LONG = [[2500, 1], [30] * 12 + [1700], [3] * 150 + [25, 2000, 0, 21]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims", [(1, 3, 64, 64), (2, 4, 128, 128)], ids=str)
@pytest.mark.parametrize("lens", LONG, ids=["2500", "1700", "2000"])
@pytest.mark.parametrize("fixed,in_place", [(True, False), (False, True)])
def test_segments(gdn, dtype, dims, lens, fixed, in_place):
    c = SlowCase(lens, dtype, *dims, fixed=fixed, seed=len(lens))
    out = prefill(gdn, c, c.pool(gdn), in_place)
    c.check(out, in_place)
    c.check_norm(out)
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims", [(1, 2, 256, 136), (2, 2, 32, 40), (1, 3, 16, 8), (1, 2, 128, 256), (3, 3, 64, 128), (1, 2, 128, 64)], ids=str)
@pytest.mark.parametrize("slow", [True, False])
def test_head_sizes(gdn, dtype, dims, slow):
    c = (SlowCase if slow else Case)([31, 700, 150], dtype, *dims, seed=dims[2])
    out = prefill(gdn, c, c.pool(gdn))
    c.check(out)
    c.check_norm(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pool_aligned_to_sixteen_bytes(gdn, dtype):
    c = SlowCase([1000, 40, 1], dtype, 1, 3, 64, 64, seed=13)
    room = torch.empty(c.state.numel() + 4, device=DEV)
    c.sd = room[4:].view(c.state.shape)
    c.sd.copy_(c.state)
    out = prefill(gdn, c, gdn.GDNStatePool(c.sd.shape[0], 1, 3, 64, 64, tensor=c.sd))
    c.check(out)
    c.check_norm(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims", [(2, 4, 128, 64), (1, 2, 64, 64), (2, 2, 32, 40)], ids=str)
@pytest.mark.parametrize("lens", [[150, 5, 300, 0, 64], [12, 20, 3]], ids=str)
def test_every_tensor_has_its_own_stride(gdn, dtype, dims, lens):
    """q, k and v at odd places of buffers of different widths, v the widest and q dense; of one token too."""
    c = Case(lens, dtype, *dims, seed=7)
    q, k, v, g = c.device_inputs()

    def inside(x, before, behind):
        T, h, d = x.shape
        room = torch.full((T, before + h * d + behind), float("nan"), dtype=x.dtype, device=DEV)
        room[:, before:before + h * d] = x.reshape(T, h * d)
        return room[:, before:before + h * d].view(T, h, d)

    q, k, v = q.contiguous(), inside(k, 8, 40), inside(v, 24, 1000)
    out = gdn.linear_attention_prefill(q, k, v, g, c.pool(gdn), i32(c.cu), i32(c.read), i32(c.write))
    c.check(out)
    c.check_norm(out)
