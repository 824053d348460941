"""The cases of slow decays see what the state carries from segment to segment: the rule with that carried wrongly, computed
here in 64 bits, is out of the tolerances of the GPU tests that use them.  No GPU."""
import pytest
import torch

from linear_helpers import SlowCase

DIMS = (1, 3, 16, 8)


def by_segments(c, span, fault):
    """Outputs and pool of the rule over segments of `span` tokens, whose states are carried with a fault."""
    hk, hv, dk, dv = c.dims
    q, k, v = (t.double() for t in c.views(c.x))
    out, pool = torch.zeros(c.T, hv, dv, dtype=torch.float64), c.state.clone().double()
    decay = torch.exp((c.decay if c.decay.dim() == 2 else c.decay.expand(c.T, hv)).double())
    head = torch.arange(hv) // (hv // hk)
    for r, n in enumerate(c.lens):
        S = c.state[c.read[r]].double()
        for s in range(0, n, span):
            start = S
            for t in range(int(c.cu[r]) + s, int(c.cu[r]) + min(s + span, n)):
                S = decay[t][:, None, None] * S + v[t][:, :, None] * k[t][head][:, None, :]
                out[t] = dk ** -0.5 * (S @ q[t][head][:, :, None])[..., 0]
            if s + span < n:
                D = torch.stack([decay[t] for t in range(int(c.cu[r]) + s, int(c.cu[r]) + s + span)]).prod(0)[:, None, None]
                own = S - D * start
                wrong = {"none": D, "dropped": 0 * D, "another head's": D.roll(1, 0),
                         "twice": D * D, "kept whole": torch.ones_like(D)}[fault]
                S = wrong * start + own
        if n:
            pool[c.write[r]] = S
        else:
            pool[c.write[r]] = c.state[c.read[r]].double()
    return out, pool.float()


@pytest.mark.parametrize("lens", [[2500, 1], [1000, 40, 1]], ids=str)
@pytest.mark.parametrize("fixed", [True, False])
def test_a_wrong_carry_is_seen(lens, fixed):
    c = SlowCase(lens, "f32", *DIMS, fixed=fixed, seed=1)
    for span in (64, 256):
        out, c.sd = by_segments(c, span, "none")
        c.check(out)
        c.check_norm(out)
        for fault in ("dropped", "another head's", "twice", "kept whole"):
            out, c.sd = by_segments(c, span, fault)
            with pytest.raises(AssertionError, match="off by"):
                c.check(out)
            with pytest.raises(AssertionError, match="norm"):
                c.check_norm(out)
