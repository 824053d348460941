"""Calls of linear attention and of attention over shared prefixes that run at the same time on two streams, each with its own
slots, outputs and workspace, and captured graphs that take turns with one workspace."""
import pytest
import torch

from attn_helpers import DEV, TYPES, i32, packed
from linear_helpers import Case
from test_gpu_shared_prefix import Forked

pytestmark = pytest.mark.gpu


def linear(G, lens, dtype, dims, seed):
    """A call over its own state pool, in place, whose outputs are its next values."""
    c = Case(lens, dtype, *dims, seed=seed)
    pool = c.pool(G)
    q, k, v, g = c.device_inputs()
    k = k * 0.1
    cu, slots = i32(c.cu), i32(c.read)
    start = c.sd.clone()

    def reset():
        c.sd.copy_(start)

    def call(times, workspace=None):
        x = v
        for _ in range(times):
            x = G.linear_attention_prefill(q, k, x, g, pool, cu, slots, keep_in_place=True, workspace=workspace)
        return x, c.sd

    return reset, call, lambda: G.linear_attention_prefill_workspace_bytes(pool, len(lens), c.T, TYPES[dtype])


def attention(G, dtype, d, seed):
    c = Forked([(40, [(9, 1), (70, 3), (0, 1), (200, 1)]), (3, [(30, 1), (5, 2)])], dtype, 2, d, 16, seed=seed)
    pool, table, lens, cu, bounds = c.pool(G), i32(c.table), i32(c.lens), i32(packed(c.new)), i32(c.bounds)
    q = torch.randn(int(sum(c.new)), 8, d, generator=torch.Generator().manual_seed(seed)).to(TYPES[dtype]).to(DEV)

    def call(times):
        x = q
        for _ in range(times):
            x = G.paged_attention_shared(x, pool, table, lens, cu, bounds, G.kv_pages_shared(table, lens, cu, bounds, 16))
        return (x,)

    return lambda: None, call


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_calls_at_once(gdn, dtype):
    work = [linear(gdn, [900, 30, 5], dtype, (2, 4, 128, 128), 1)[:2], linear(gdn, [5, 1500], dtype, (2, 2, 64, 64), 2)[:2],
            attention(gdn, dtype, 128, 3), attention(gdn, dtype, 64, 4)]
    alone = []
    for reset, call in work:
        reset()
        alone.append([x.clone() for x in call(20)])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(5):
        for reset, _ in work:
            reset()
        torch.cuda.synchronize()
        together = []
        for stream, (_, call) in zip(streams, work):
            with torch.cuda.stream(stream):
                together.append(call(20))
        torch.cuda.synchronize()
        for a, b in zip(alone, together):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graphs_that_take_turns_with_a_workspace(gdn, dtype):
    calls = [linear(gdn, [1500, 3], dtype, (1, 2, 64, 64), 5), linear(gdn, [1400, 200], dtype, (1, 2, 64, 64), 6)]
    workspace = torch.full((max(need() for _, _, need in calls),), 255, dtype=torch.uint8, device=DEV)
    want, graphs = [], []
    for reset, call, _ in calls:
        reset()
        want.append([x.clone() for x in call(1)])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call(1, workspace)
        graphs.append((graph, got))
    for _ in range(4):
        for reset, _, _ in calls:
            reset()
        for graph, _ in graphs:
            graph.replay()
        for a, (_, b) in zip(want, graphs):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
