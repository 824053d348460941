"""Helpers for the tests of the attention layers over a paged cache: scattered
pages, and the operators' definitions in 64 bits on the CPU.

Tolerances (written here, used by every parity test), with A = sum_j w_j |v_j|
the magnitude of the terms of an output, w the softmax weights:
  * bf16 attention: 2^-8 |o| for the output's rounding (bf16 has eight significant
    bits, so rounding to nearest is off by up to 2^-8 of the value), and 2^-8 A:
    every weight is rounded to bf16 once
  * f32 attention: 4e-5 A.  A score is an fp32 sum of d products: its error is
    about 2^-24 sqrt(d) sum |q k| scale, 2e-5 at d = 256 with terms of order 1,
    and it multiplies the weight
  * prologue: a value takes about ten fp32 operations (the norm's sum of squares
    by pairs among them), 2^-20 of the largest term, then one rounding to bf16 (2^-8)
"""
import numpy as np
import torch

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(np.asarray(a, dtype=np.int32)), device=DEV)


class Cache:
    """Rows of given lengths on scattered pages of a random pool; `poison` fills
    every place that no row's token holds (the null page too)."""

    def __init__(self, lens, dtype, hkv, d, page, layers=1, spare=3, seed=0, poison=None, max_pages=None):
        rng = np.random.default_rng(seed)
        self.lens, self.dtype, self.hkv, self.d, self.page, self.layers = list(lens), dtype, hkv, d, page, layers
        held = [-(-n // page) for n in lens]
        self.num_pages = 1 + sum(held) + spare
        order = 1 + rng.permutation(self.num_pages - 1)
        self.max_pages = max_pages or max(held + [1])
        self.table = np.zeros((len(lens), self.max_pages), np.int32)
        at = 0
        for r, n in enumerate(held):
            self.table[r, :n] = order[at:at + n]
            at += n
        shape = (layers, self.num_pages, hkv, page, d)
        g = torch.Generator().manual_seed(seed)
        self.k = torch.randn(shape, generator=g).to(TYPES[dtype])
        self.v = torch.randn(shape, generator=g).to(TYPES[dtype])
        if poison is not None:
            held_places = torch.zeros(shape[1], page, dtype=torch.bool)
            for r, n in enumerate(lens):
                for j in range(n):
                    held_places[self.table[r, j // page], j % page] = True
            for x in (self.k, self.v):
                x.permute(0, 2, 1, 3, 4)[:, :, ~held_places] = poison

    def pool(self, G):
        self.kd, self.vd = self.k.to(DEV), self.v.to(DEV)
        return G.KVPagePool(self.num_pages, self.page, self.hkv, self.d, layers=self.layers, dtype=TYPES[self.dtype],
                            k=self.kd, v=self.vd)

    def keys(self, r, layer=0):
        """K and V of row r, [hkv][len][d], in 64 bits."""
        n = self.lens[r]
        pages = torch.as_tensor(self.table[r, : -(-n // self.page)].astype(np.int64))
        return [x[layer][pages].transpose(0, 1).reshape(self.hkv, -1, self.d)[:, :n].double() for x in (self.k, self.v)]


def packed(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def attention_ref(c, q, new, scale, layer=0):
    """(out, A) of q [T][hq][d], in 64 bits; padding rows and rows without tokens give zeros."""
    T, hq, d = q.shape
    g = hq // c.hkv
    out, mag = torch.zeros(T, hq, d, dtype=torch.float64), torch.zeros(T, hq, d, dtype=torch.float64)
    t = 0
    for r, n in enumerate(new):
        if c.lens[r] and n:
            k, v = c.keys(r, layer)
            for i in range(n):
                see = c.lens[r] - n + i + 1
                x = q[t + i].double().view(c.hkv, g, d)
                w = torch.softmax(torch.einsum("hgd,hjd->hgj", x, k[:, :see]) * scale, -1)
                out[t + i] = torch.einsum("hgj,hjd->hgd", w, v[:, :see]).reshape(hq, d)
                mag[t + i] = torch.einsum("hgj,hjd->hgd", w, v[:, :see].abs()).reshape(hq, d)
        t += n
    return out, mag


def check_attention(out, ref, mag, dtype):
    o = out.double().cpu()
    tol = 2.0 ** -8 * (ref.abs() + mag) if dtype == "bf16" else 4e-5 * mag
    assert torch.isfinite(o).all()
    worst = ((o - ref).abs() - tol).max().item()
    assert worst <= 0, f"out of tolerance by {worst:.3g} (largest error {(o - ref).abs().max().item():.3g})"


def prologue_ref(x, w, eps, rope, pos, rot, interleaved):
    """(y, magnitude of its terms) of heads x [heads][d] of one token, in 64 bits."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    y, mag = x.clone(), x.abs().clone()
    half = rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = rope[pos, i].double(), rope[pos, half + i].double()
        y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
        mag[:, a] = mag[:, b] = x[:, a].abs() + x[:, b].abs()
    return y, mag


def check_prologue(got, ref, mag, dtype):
    tol = 2.0 ** -20 * mag + (2.0 ** -8 * ref.abs() if dtype == "bf16" else 0.0)
    err = (got.double().cpu() - ref).abs()
    assert (err <= tol).all(), f"largest error {err.max().item():.3g}"
