"""Helpers for the tests of linear attention with a decay for each head: inputs, and the rule in 64 bits on the CPU.

Tolerances (written here, used by every parity test).  `reference` also returns magnitudes: of the state, M' = e^g M + |v| |k|
from M = |S|, and of an output, A = scale sum M |q|, the sums of the terms' absolute values.
  * state: a step multiplies by e^g (off by at most 2^-22 of it, expf's two units and the product's rounding) and adds v k
    with one rounding, so n steps are off by at most n 2^-21 M; the chunked form adds the same terms in another order, each
    weighted by one exponential whose argument is off by 2^-24 of a sum of at most 128 decays: within the same bound for n + 8
  * fp32 output: the state's error in every term, and the sum over dk <= 256 terms in runs of 16: (n + 8) 2^-21 A
  * bf16 output: 2^-8 |o| for its own rounding; the chunked form also rounds the weights of the chunk's own tokens and the state
    that it multiplies with q to bf16, each 2^-8 of its terms, together at most 2^-8 A
"""
import numpy as np
import torch

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(np.asarray(a, dtype=np.int32)), device=DEV)


class Case:
    """Packed sequences (a batch of single tokens: lengths of one) with states on scattered slots; every third slot of the
    pool is nobody's.  pad: sequences on slot 0."""

    def __init__(self, lens, dtype, hk, hv, dk, dv, fixed=False, pad=(), seed=0, behind=0, strong=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.dtype, self.dims = list(lens), dtype, (hk, hv, dk, dv)
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        self.T = T = int(self.cu[-1]) + behind
        # a packed projection with a few columns of something else behind it
        self.x = torch.randn(T, 2 * hk * dk + hv * dv + 8, generator=g).to(TYPES[dtype])
        self.decay = -torch.rand(hv if fixed else (T, hv), generator=g) * (3.0 if strong else 0.3)
        rng = np.random.default_rng(seed)
        n = len(lens)
        order = 1 + rng.permutation(3 * n)
        self.read, self.write = order[:n].astype(np.int32), order[n:2 * n].astype(np.int32)
        self.pad = set(pad)
        for r in self.pad:
            self.read[r] = self.write[r] = 0
        self.state = torch.randn(3 * n + 1, hv, dv, dk, generator=g)
        self.state[0] = 0

    def views(self, x):
        hk, hv, dk, dv = self.dims
        T, a, b = x.shape[0], hk * dk, 2 * hk * dk
        return x[:, :a].view(T, hk, dk), x[:, a:b].view(T, hk, dk), x[:, b:b + hv * dv].view(T, hv, dv)

    def pool(self, G):
        hk, hv, dk, dv = self.dims
        self.sd = self.state.to(DEV)
        return G.GDNStatePool(self.sd.shape[0], hk, hv, dk, dv, tensor=self.sd)

    def device_inputs(self):
        return (*self.views(self.x.to(DEV)), self.decay.to(DEV))

    def reference(self, scale=None):
        """(outputs, their magnitudes A, states by sequence, their magnitudes M)"""
        hk, hv, dk, dv = self.dims
        scale = dk ** -0.5 if scale is None else scale
        q, k, v = (t.double() for t in self.views(self.x))
        head = torch.arange(hv) // (hv // hk)
        out, mag = torch.zeros(self.T, hv, dv, dtype=torch.float64), torch.zeros(self.T, hv, dv, dtype=torch.float64)
        states, mags = [], []
        for r, n in enumerate(self.lens):
            S = self.state[self.read[r]].double()
            M = S.abs()
            if r not in self.pad:
                for t in range(self.cu[r], self.cu[r] + n):
                    a = torch.exp((self.decay if self.decay.dim() == 1 else self.decay[t]).double().clamp(max=0))[:, None, None]
                    kt, qt = k[t][head], q[t][head]
                    S = a * S + v[t][:, :, None] * kt[:, None, :]
                    M = a * M + (v[t][:, :, None] * kt[:, None, :]).abs()
                    out[t] = scale * (S @ qt[:, :, None])[..., 0]
                    mag[t] = abs(scale) * (M @ qt.abs()[:, :, None])[..., 0]
            states.append(S)
            mags.append(M)
        return out, mag, states, mags

    def check(self, out, in_place=False, scale=None, bits=None):
        """Outputs and the whole pool against the reference; slots that nobody writes bit for bit."""
        ref, A, states, mags = self.reference(scale)
        last = int(self.cu[-1])
        o, n = out.double().cpu()[:last], max(self.lens + [0])
        bound = (n + 8) * 2.0 ** -21 * A[:last]
        if self.dtype == "bf16":
            bound = bound + 2.0 ** -8 * ref[:last].abs() + 2.0 ** -8 * A[:last]
        assert torch.isfinite(o).all()
        worst = ((o - ref[:last]).abs() - bound).max() if last else torch.tensor(-1.0)
        assert worst <= 0, f"outputs off by {worst} over the bound"
        pool, want = self.sd.cpu(), self.state.clone()
        for r in range(len(self.lens)):
            if r in self.pad:
                continue
            slot = self.read[r] if in_place else self.write[r]
            off = (pool[slot].double() - states[r]).abs() - (self.lens[r] + 8) * 2.0 ** -21 * mags[r]
            assert off.max() <= 0, f"state of sequence {r} off by {off.max()} over the bound"
            want[slot] = pool[slot]
        assert torch.equal(pool, want), "a slot that nobody writes changed"

    def check_norm(self, out, scale=None):
        """Of every sequence of more than 20 tokens and head, the difference's norm over the output's.

        bf16: the weights, the state as a factor, and the output are rounded, each value by at most half a step, which is spread
        evenly over +- 2^-8 of it at worst, 2^-8 / sqrt(3) = 0.00226 in the mean square.  The terms of an output have random
        signs, so what the first two give has at most the output's own norm times that: sqrt(2) 0.00226 = 0.0032 in all.  The
        rest of the limit of 0.004 is for the spread of a norm over some thousands of values.
        fp32: a product leaves out 2^-22 of a term and a sum of sixteen is cut short by up to 2^-21 of it, an exponential is off by
        2^-22 and a state's step by 2^-24: 2^-19 with the same random signs."""
        ref = self.reference(scale)[0]
        limit = 0.004 if self.dtype == "bf16" else 2.0 ** -19
        o = out.double().cpu()
        for r, n in enumerate(self.lens):
            if n > 20 and r not in self.pad:
                at = slice(int(self.cu[r]), int(self.cu[r + 1]))
                off = (o[at] - ref[at]).pow(2).sum((0, 2)).sqrt() / ref[at].pow(2).sum((0, 2)).sqrt()
                assert off.max() <= limit, f"sequence {r}: off by {off.tolist()} of the outputs' norm"


class SlowCase(Case):
    """A memory of 1,000 to 10,000 tokens, another one a head, and a head that keeps all (every third): the state from before a
    segment of some hundreds of tokens is most of the one after it."""

    def __init__(self, lens, dtype, hk, hv, dk, dv, fixed=False, seed=0, **k):
        super().__init__(lens, dtype, hk, hv, dk, dv, fixed=fixed, seed=seed, **k)
        rate = 10.0 ** (-4 + torch.arange(hv).float() / max(hv - 1, 1))
        rate[2::3] = 0.0
        step = torch.ones(hv) if fixed else 0.5 + torch.rand(self.T, hv, generator=torch.Generator().manual_seed(seed + 1))
        self.decay = -rate * step
