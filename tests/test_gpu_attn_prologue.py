"""attn_prologue and rope_table on the GPU against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

from attn_helpers import DEV, TYPES, Cache, check_prologue, i32, packed, prologue_ref

pytestmark = pytest.mark.gpu


def rope(positions, rot, base=10000.0):
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def check(gdn, dtype, hq, hkv, d, rot, interleaved, new, lens, page=16, norms=(True, True), seed=0, layers=1, layer=0):
    c = Cache(lens, dtype, hkv, d, page, seed=seed, layers=layers)
    T, width = sum(new), (hq + 2 * hkv) * d
    g = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(T, width, generator=g).mul(1.5).to(TYPES[dtype])
    t = 0
    for r, n in enumerate(new):  # padding tokens hold anything
        if lens[r] == 0:
            x[t:t + n] = float("nan")
        t += n
    w = [1 + 0.3 * torch.randn(d, generator=g) if on else None for on in norms]
    table = rope(max(lens) + 1, rot) if rot else None
    pool = c.pool(gdn)
    xd = x.to(DEV)
    cut = lambda y: (y[:, :hq * d].view(T, hq, d), y[:, hq * d:(hq + hkv) * d].view(T, hkv, d),  # noqa: E731
                     y[:, (hq + hkv) * d:].view(T, hkv, d))
    out = gdn.attn_prologue(*cut(xd), pool, table.to(DEV) if rot else None, i32(c.table), i32(lens), i32(packed(new)),
                            layer=layer, q_norm=w[0].to(DEV) if norms[0] else None,
                            k_norm=w[1].to(DEV) if norms[1] else None, eps=1e-5, interleaved=interleaved)
    assert gdn.get_device_error() == 0
    q, k, v = cut(x)
    written = torch.zeros(c.k.shape[:2] + (page,), dtype=torch.bool)
    kd, vd = c.kd.cpu(), c.vd.cpu()
    t = 0
    for r, n in enumerate(new):
        for i in range(n):
            if lens[r] == 0:
                assert (out[t + i] == 0).all()
                continue
            p = lens[r] - n + i
            at = (layer, int(c.table[r, p // page]), slice(None), p % page)
            check_prologue(out[t + i], *prologue_ref(q[t + i], w[0], 1e-5, table, p, rot, interleaved), dtype)
            check_prologue(kd[at], *prologue_ref(k[t + i], w[1], 1e-5, table, p, rot, interleaved), dtype)
            assert torch.equal(vd[at], v[t + i])
            written[layer, at[1], p % page] = True
        t += n
    keep = ~written[:, :, None, :, None].expand_as(c.k)
    assert torch.equal(kd[keep], c.k[keep]) and torch.equal(vd[keep], c.v[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot", [(4, 4, 64, 64), (12, 4, 64, 16), (16, 4, 128, 128), (7, 1, 128, 96), (16, 2, 256, 64),
                                          (6, 2, 256, 256), (3, 3, 64, 48), (40, 8, 128, 32)])
def test_heads_and_rotations(gdn, dtype, interleaved, hq, hkv, d, rot):
    check(gdn, dtype, hq, hkv, d, rot, interleaved, [1, 3, 1, 20, 0, 1], [1, 17, 0, 20, 9, 333])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norms", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("rot", [0, 64])
def test_norms_and_no_rotation(gdn, dtype, norms, rot):
    check(gdn, dtype, 4, 2, 128, rot, False, [2, 5], [40, 5], norms=norms)


def test_many_tokens_and_layers(gdn):
    check(gdn, "bf16", 4, 2, 64, 64, False, [700, 1, 1300], [900, 50, 1300], page=64, layers=3, layer=1)


def test_rows_by_the_thousand(gdn):
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 50, 1100).tolist()
    check(gdn, "f32", 2, 1, 64, 32, True, [min(n, 1) if r % 3 else min(n, 2) for r, n in enumerate(lens)], lens)


def test_in_place(gdn):
    c = Cache([300, 40], "bf16", 2, 64, 16, seed=9)
    q = torch.randn(270, 4, 64, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    k = torch.randn(270, 2, 64).bfloat16().to(DEV)
    args = (k, k, c.pool(gdn), rope(300, 32).to(DEV), i32(c.table), i32(c.lens), i32([0, 250, 270]))
    want = gdn.attn_prologue(q, *args)
    assert gdn.attn_prologue(q, *args, out=q) is q
    assert torch.equal(q, want)


def test_bad_tokens_are_left_out(gdn):
    """A row shorter than its tokens, a position past the rotation table, bad pages, tokens outside every row."""
    lens, new = [30, 1, 100, 20, 16], [2, 3, 1, 1, 2]
    c = Cache([30, 3, 100, 20, 16], "f32", 2, 64, 16, seed=2)
    T = 11  # the last two tokens belong to no row
    x = torch.randn(T, 4, 64, generator=torch.Generator().manual_seed(4))
    table = c.table.copy()
    table[3, 1] = c.num_pages
    pool = c.pool(gdn)
    r = rope(64, 64).to(DEV)
    k, v = x[:, :2].contiguous(), x[:, 2:].contiguous()
    out = gdn.attn_prologue(x.to(DEV), k.to(DEV), v.to(DEV), pool, r, i32(table), i32(lens), i32(packed(new)))
    assert gdn.get_device_error() == gdn.GDN_DEVERR_BAD_PAGE
    dead = [2, 3, 4, 5, 6, 9, 10]
    assert (out[dead] == 0).all()
    kd, vd = c.kd.cpu(), c.vd.cpu()
    changed = (kd != c.k).any(-1).any(2)[0] | (vd != c.v).any(-1).any(2)[0]
    places = {(int(c.table[0, p // 16]), p % 16) for p in (28, 29)} | {(int(c.table[4, 0]), p) for p in (14, 15)}
    assert {tuple(i) for i in changed.nonzero().tolist()} == places
    for t, p in ((0, 28), (1, 29), (7, 14), (8, 15)):
        check_prologue(out[t], *prologue_ref(x[t], None, 0, r.cpu(), p, 64, False), "f32")


def test_wrong_arguments_are_refused(gdn):
    c = Cache([20], "bf16", 2, 128, 16)
    pool, table, lens, cu = c.pool(gdn), i32(c.table), i32(c.lens), i32([0, 1])
    z = lambda h: torch.zeros(1, h, 128, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    r = rope(32, 64).to(DEV)
    go = lambda q=z(4), k=z(2), v=z(2), r=r, **kw: gdn.attn_prologue(q, k, v, pool, r, table, lens, cu, **kw)  # noqa: E731
    go()
    for bad in (dict(q=z(4).float()), dict(r=r.half())):
        with pytest.raises(TypeError):
            go(**bad)
    for bad in (dict(k=z(1)), dict(k=z(2)[:0]), dict(q_norm=torch.ones(64, device=DEV)), dict(q=z(4).cpu()),
                dict(q=torch.zeros(1, 128, 4, dtype=torch.bfloat16, device=DEV).transpose(1, 2))):
        with pytest.raises(ValueError):
            go(**bad)
    for bad in (dict(q=z(3)), dict(r=rope(32, 8).to(DEV)), dict(r=torch.zeros(4, 144, device=DEV)), dict(layer=-1),
                dict(q_norm=torch.ones(128, device=DEV), eps=float("nan")),
                dict(q=torch.zeros(4 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(1, 4, 128))):
        with pytest.raises(gdn.GDNError):
            go(**bad)


@pytest.mark.parametrize("scaling", [None, {"type": "linear", "factor": 4}, {"type": "ntk", "factor": 8},
                                     {"type": "yarn", "factor": 4, "original": 4096}])
def test_rope_table(gdn, scaling):
    """Against 64 bits: an fp32 entry is off by half a unit of its last place, 2^-25 for values up to one, and mscale adds
    one rounding; 64-bit sines of angles up to 2e5 are exact to 1e-10."""
    rot, positions = 64, 200001
    t = gdn.rope_table(rot, positions, base=1e6, scaling=scaling).cpu().double()
    freq, m = gdn.rope_inv_freq(rot, 1e6, scaling)
    for p in (0, 1, 2, 4095, 65537, 200000):
        a = p * freq
        want = torch.cat([a.cos(), a.sin()]) * m
        assert (t[p] - want).abs().max() <= m * 2.0 ** -24


def test_rope_scalings_of_a_known_case(gdn):
    plain, one = gdn.rope_inv_freq(128, 10000.0)
    assert one == 1.0 and plain[0] == 1.0
    assert torch.allclose(gdn.rope_inv_freq(128, 10000.0, {"type": "linear", "factor": 4})[0] * 4, plain, rtol=1e-15)
    ntk = gdn.rope_inv_freq(128, 10000.0, {"type": "ntk", "factor": 4})[0]
    assert ntk[0] == 1.0 and abs(ntk[-1] * 4 / plain[-1] - 1) < 1e-12
    y, m = gdn.rope_inv_freq(128, 10000.0, {"type": "yarn", "factor": 16, "original": 4096})
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(y[turns > 34], plain[turns > 34])
    assert torch.allclose(y[turns < 0.9], plain[turns < 0.9] / 16, rtol=1e-12)
    assert abs(m - (0.1 * math.log(16) + 1)) < 1e-12
