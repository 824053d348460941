"""Linear attention with a decay for each head, decode and prefill, against the rule in 64 bits."""
import math

import pytest
import torch

from linear_helpers import DEV, TYPES, Case, i32

pytestmark = pytest.mark.gpu

SHAPES = [(2, 2, 128, 128), (1, 3, 64, 64), (2, 4, 128, 64), (1, 2, 64, 128), (2, 2, 16, 8), (1, 2, 32, 40), (1, 1, 256, 136)]


def decode(G, c, pool, in_place=False, **k):
    q, kk, v, g = c.device_inputs()
    return G.linear_attention_decode(q, kk, v, g, pool, i32(c.read), None if in_place else i32(c.write), keep_in_place=in_place, **k)


def prefill(G, c, pool, in_place=False, **k):
    q, kk, v, g = c.device_inputs()
    return G.linear_attention_prefill(q, kk, v, g, pool, i32(c.cu), i32(c.read), None if in_place else i32(c.write),
                                      keep_in_place=in_place, **k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("fixed,in_place", [(True, False), (False, True)])
def test_decode(gdn, dtype, shape, fixed, in_place):
    c = Case([1] * 5, dtype, *shape, fixed=fixed, pad=[1], seed=1)
    c.check(decode(gdn, c, c.pool(gdn), in_place), in_place)
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("rows", [0, 1, 2, 33])
def test_decode_rows(gdn, rows):
    c = Case([1] * rows, "bf16", 2, 4, 128, 128, seed=rows)
    out = decode(gdn, c, c.pool(gdn), scale=0.3)
    c.check(out, scale=0.3)
    assert out.shape == (rows, 4, 128)


LENS = [[1], [3, 0, 1, 9, 17], [0], [40, 1, 64], [127], [128], [129, 33], [300, 2, 257]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_prefill_shapes(gdn, dtype, shape):
    c = Case([150, 5, 0, 66], dtype, *shape, pad=[1], seed=2)
    c.check(prefill(gdn, c, c.pool(gdn)))
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("fixed,in_place", [(True, True), (False, False)])
def test_prefill_lengths(gdn, dtype, lens, fixed, in_place):
    c = Case(lens, dtype, 1, 2, 128, 128, fixed=fixed, seed=len(lens), strong=not fixed)
    c.check(prefill(gdn, c, c.pool(gdn), in_place), in_place)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_long_sequence(gdn, dtype):
    """Long enough to be cut along its tokens, where the kernels do that."""
    c = Case([2500, 1], dtype, 1, 1, 64, 64, seed=3)
    c.check(prefill(gdn, c, c.pool(gdn)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims", [(1, 2, 64, 64), (1, 1, 128, 128)], ids=str)
@pytest.mark.parametrize("lens", [[1] * 24 + [300], [30] * 12 + [1700], [3] * 150 + [25, 2000, 0, 21]], ids=["300", "1700", "2000"])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_long_sequence_among_short_ones(gdn, dtype, dims, lens, in_place):
    """The mean, which is all that the host knows, says there are no chunks, or that no sequence is cut."""
    c = Case(lens, dtype, *dims, pad=[0, 3], seed=5)
    c.check(prefill(gdn, c, c.pool(gdn), in_place), in_place)
    assert gdn.get_device_error() == 0


def test_decays_at_their_ends(gdn):
    """-inf forgets what came before, 0 and what is above keep all of it."""
    for dtype in ("bf16", "f32"):
        c = Case([200, 40], dtype, 1, 2, 64, 64, seed=4)
        c.decay[50, 0] = c.decay[170, 1] = c.decay[199, 0] = -math.inf
        c.decay[60:70] = 0.0
        c.decay[100:110] = 0.5
        c.decay[210:215] = -1e30
        c.check(prefill(gdn, c, c.pool(gdn)))
    c = Case([1] * 4, "f32", 1, 2, 64, 64, seed=4)
    c.decay[1], c.decay[2], c.decay[3] = -math.inf, 0.0, 2.0
    c.check(decode(gdn, c, c.pool(gdn)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_values_that_are_not_finite_stay_where_they_are(gdn, dtype, where):
    """A NaN or infinity at a token reaches its own sequence from there on (q: its own token only) and nothing else."""
    bad = 100
    for value in (math.nan, math.inf):
        c = Case([60, 190, 20], dtype, 1, 2, 128, 128, seed=5)
        clean = prefill(gdn, c, c.pool(gdn)).float()
        states = c.sd.clone()
        views = dict(zip("qkv", c.views(c.x)))
        views[where][bad, 0, 3] = value
        out = prefill(gdn, c, c.pool(gdn)).float()
        same = torch.ones(c.T, dtype=torch.bool)
        same[bad:(bad + 1 if where == "q" else 250)] = False
        assert torch.equal(out[same], clean[same])
        assert not torch.isfinite(out[bad, 0]).all()
        if where == "v":  # one element of the first head's values
            assert torch.equal(out[:, 1], clean[:, 1])
            keep = torch.arange(128) != 3
            assert torch.equal(out[:, 0, keep], clean[:, 0, keep])
            assert not torch.isfinite(out[bad:250, 0, 3]).any()
        mine = int(c.write[1])
        others = [s for s in range(len(states)) if s != mine]
        assert torch.equal(c.sd[others], states[others])
        if where == "q":
            assert torch.equal(c.sd[mine], states[mine])
        else:
            assert not torch.isfinite(c.sd[mine, 0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_behind_the_last_sequence_are_left_alone(gdn, dtype):
    c = Case([130, 4], dtype, 1, 2, 128, 128, seed=6, behind=30)
    for x in c.views(c.x):
        x[134:] = math.nan
    out = torch.full((c.T, 2, 128), 7.0, dtype=TYPES[dtype], device=DEV)
    assert prefill(gdn, c, c.pool(gdn), out=out) is out
    c.check(out)
    assert (out[134:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pool_aligned_to_sixteen_bytes(gdn, dtype):
    """A wrapped pool's memory need not be aligned to more."""
    c = Case([1000, 40, 1], dtype, 1, 1, 64, 64, seed=13)
    room = torch.empty(c.state.numel() + 4, device=DEV)
    c.sd = room[4:].view(c.state.shape)
    assert c.sd.data_ptr() % 32 == 16
    c.sd.copy_(c.state)
    c.check(prefill(gdn, c, gdn.GDNStatePool(c.sd.shape[0], 1, 1, 64, 64, tensor=c.sd)))
    d = Case([1] * 3, dtype, 1, 1, 64, 64, seed=14)
    d.sd = room[4:4 + d.state.numel()].view(d.state.shape)
    d.sd.copy_(d.state)
    d.check(decode(gdn, d, gdn.GDNStatePool(d.sd.shape[0], 1, 1, 64, 64, tensor=d.sd)))


def test_prefill_is_decode_token_after_token(gdn):
    """fp32, and tokens of a sequence fed in two calls."""
    c = Case([37], "f32", 2, 2, 64, 64, seed=7)
    pool = c.pool(gdn)
    q, k, v, g = c.device_inputs()
    whole = prefill(gdn, c, pool)
    other = torch.zeros_like(c.sd)
    other[1] = c.sd[int(c.read[0])]
    step = gdn.GDNStatePool(other.shape[0], 2, 2, 64, 64, tensor=other)
    a, b = [1, 2], []
    for t in range(37):
        b.append(gdn.linear_attention_decode(q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], step, i32(a[:1]), i32(a[1:])))
        a.reverse()
    # the same sums; the products' order may differ by form, so to rounding: 37 steps of 2^-21
    assert (torch.cat(b) - whole).abs().max() <= 45 * 2.0 ** -21 * c.reference()[1].max()


def test_bad_slots(gdn):
    c = Case([1] * 4, "bf16", 1, 2, 64, 64, seed=8)
    pool = c.pool(gdn)
    before = c.sd.clone()
    read, write = c.read.copy(), c.write.copy()
    read[0], write[1], write[2] = len(before), 0, read[2]
    q, k, v, g = c.device_inputs()
    for call in (lambda: gdn.linear_attention_decode(q, k, v, g, pool, i32(read), i32(write)),
                 lambda: gdn.linear_attention_prefill(q, k, v, g, pool, i32(c.cu), i32(read), i32(write))):
        out = call()
        assert gdn.get_device_error() == gdn.GDN_DEVERR_BAD_SLOT
        assert (out[:3] == 0).all() and (out[3] != 0).any()
        changed = (c.sd != before).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed == [int(c.write[3])]
        c.sd.copy_(before)


def test_bad_ranges(gdn):
    """cu_seqlens that go backwards or out of the tokens: those sequences are skipped, nothing is written outside."""
    c = Case([10, 10, 10], "bf16", 1, 1, 128, 128, seed=9)
    pool = c.pool(gdn)
    before = c.sd.clone()
    q, k, v, g = c.device_inputs()
    out = torch.full((30, 1, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    gdn.linear_attention_prefill(q, k, v, g, pool, i32([-4, 10, 5, 40]), i32(c.read), i32(c.write), out=out)
    assert gdn.get_device_error() == gdn.GDN_DEVERR_BAD_SLOT
    assert (out == 7).all() and torch.equal(c.sd, before)


def test_captured_and_on_another_stream(gdn):
    for make, call in ((lambda s: Case([1] * 6, "bf16", 2, 2, 128, 128, seed=s), decode),
                       (lambda s: Case([200, 7, 33], "bf16", 2, 2, 128, 128, seed=s), prefill)):
        c = make(10)
        call(gdn, c, c.pool(gdn))  # (the error word is found by now)
        pool = c.pool(gdn)
        x, decay = c.x.to(DEV), c.decay.to(DEV)
        q, k, v = c.views(x)
        cu, read, write = i32(c.cu), i32(c.read), i32(c.write)
        run = ((lambda: gdn.linear_attention_decode(q, k, v, decay, pool, read, write)) if call is decode else
               (lambda: gdn.linear_attention_prefill(q, k, v, decay, pool, cu, read, write)))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        d = make(11)
        d.read, d.write = c.read, c.write
        x.copy_(d.x)
        decay.copy_(d.decay)
        d.sd = c.sd
        c.sd.copy_(d.state)
        graph.replay()
        torch.cuda.synchronize()
        d.check(out)
        again = out.clone()
        c.sd.copy_(d.state)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = run()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(other, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[700], [5, 300, 1, 90]], ids=str)
def test_calls_behind_one_another(gdn, dtype, lens):
    """The kernels of a call run beside each other and are launched before those ahead of them end: calls that each read what
    the one before wrote (states in place, values) give the same bits with and without a pause between them."""
    c = Case(lens, dtype, 2, 2, 64, 64)
    q, k, v, g = c.device_inputs()
    cu, slots, one = i32(c.cu), i32(c.read), i32(c.read[:1])
    k = k * 0.1

    def run(pool, pause):
        x, outs = v.clone(), []
        for _ in range(12):
            x = gdn.linear_attention_prefill(q, k, x, g, pool, cu, slots, keep_in_place=True)
            pause()
            outs.append(gdn.linear_attention_decode(q[:1], k[:1], x[:1], g[:1], pool, one, keep_in_place=True))
            pause()
        return torch.cat([o.flatten() for o in outs] + [x.flatten()])

    a = run(c.pool(gdn), torch.cuda.synchronize)
    s = c.sd
    assert torch.isfinite(a).all()
    for _ in range(3):
        b = run(c.pool(gdn), lambda: None)
        assert torch.equal(a, b) and torch.equal(s, c.sd)
    pool = c.pool(gdn)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = run(pool, lambda: None)
    for _ in range(3):
        c.sd.copy_(c.state)
        graph.replay()
        assert torch.equal(a, b) and torch.equal(s, c.sd)


def test_python_refusals(gdn):
    c = Case([3, 2], "bf16", 1, 2, 64, 64)
    pool = c.pool(gdn)
    q, k, v, g = c.device_inputs()
    cu, read, write = i32(c.cu), i32(c.read), i32(c.write)

    def call(**x):
        a = dict(q=q, k=k, v=v, log_decay=g, pool=pool, cu_seqlens=cu, read_slot=read, write_slot=write)
        a.update(x)
        gdn.linear_attention_prefill(**a)

    call()
    with pytest.raises(ValueError, match="more than a call takes"):
        call(q=q[:1].expand(2 ** 31, -1, -1))
    for wrong in (dict(q=q[:, :, :32]), dict(k=k[:4]), dict(v=v.transpose(1, 2)), dict(log_decay=g[:, :1]), dict(log_decay=g[None]),
                  dict(read_slot=read[:1]), dict(q=q.cpu()), dict(out=torch.empty(4, 2, 64, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises((ValueError, gdn.GDNError)):
            call(**wrong)
    for wrong in (dict(k=k.float()), dict(q=q.half(), k=k.half(), v=v.half()), dict(log_decay=g.double()), dict(read_slot=read.long())):
        with pytest.raises(TypeError):
            call(**wrong)
    with pytest.raises(gdn.GDNError):
        call(write_slot=None)
    with pytest.raises(gdn.GDNError):
        call(scale=math.inf)


@pytest.mark.parametrize("op", ["decode", "prefill"])
def test_both_bindings_make_the_same_calls(gdn, monkeypatch, op):
    from gated_deltanet_decode_gb300 import _lib
    if _lib.fast() is None:
        pytest.skip("the C++ binding was not built")
    results = []
    for way in range(2):
        c = Case([1] * 3 if op == "decode" else [140, 3], "bf16", 1, 2, 64, 64, seed=12)
        pool = c.pool(gdn)
        assert bool(pool._p) == (way == 0)
        call = decode if op == "decode" else prefill
        results.append((call(gdn, c, pool), c.sd.clone(), call(gdn, c, c.pool(gdn), True), c.sd))
        monkeypatch.setattr(_lib, "_fast", None)
    for x, y in zip(*results):
        assert torch.equal(x, y)
