"""Linear attention where one element of an input has the largest finite value of its type: against the rule in 64 bits, in
which it reaches the tokens that see it, as itself, and no others.

What multiplies the element is made small (2^-10), so that every term of the rule, and every weight and product of the chunked
form, stays within the range; the tolerances are those of linear_helpers, relative to the terms' absolute values, and hold
whatever those are.  The element leaves tokens and columns that do not see it as they are."""
import pytest
import torch

from linear_helpers import TYPES, Case
from test_gpu_linear_attention import decode, prefill

pytestmark = pytest.mark.gpu

SMALL = 2.0 ** -10


def with_top(c, where, tok, el, sign):
    """The element `el` of a head, at token `tok`."""
    q, k, v = c.views(c.x)
    top = sign * torch.finfo(TYPES[c.dtype]).max
    if where == "v":  # S' gets v k
        v[tok, :, el] = top
        k[tok] *= SMALL
    elif where == "k":  # S' gets v k, outputs and weights get k q
        k[tok, :, el] = top
        v[tok] *= SMALL
        q[:, :, el] *= SMALL
    else:  # outputs get S q, weights k q; the state's column comes from k's
        q[tok, :, el] = top
        k[:, :, el] *= SMALL
        c.state[1:, :, :, el] *= SMALL


DIMS = [(1, 2, 64, 64), (1, 1, 128, 128), (1, 2, 128, 64), (2, 2, 32, 40), (1, 1, 256, 136)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("where", ["v", "k", "q"])
@pytest.mark.parametrize("lens,tok", [([100, 5, 30], 10), ([100, 5, 30], 40), ([100, 5, 30], 103), ([700], 130), ([700], 699)], ids=str)
def test_largest_finite_values(gdn, dtype, dims, where, lens, tok):
    c = Case(lens, dtype, *dims, seed=tok)
    with_top(c, where, tok, 3, -1 if tok % 4 else 1)
    c.check(prefill(gdn, c, c.pool(gdn)))
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("lens", [[100, 5], [700]], ids=str)
def test_largest_finite_values_of_the_state(gdn, dtype, dims, lens):
    """(Of bf16's range with bf16 activations, where the state is a factor of the outputs in bf16.)"""
    c = Case(lens, dtype, *dims, seed=3)
    top = torch.finfo(TYPES[dtype]).max
    q, k, v = c.views(c.x)
    q[:, :, 5] *= SMALL
    c.state[1:, :, 2, 5] = top
    c.state[1:, :, 7, 5] = -top
    c.check(prefill(gdn, c, c.pool(gdn)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["v", "k", "q"])
def test_largest_finite_values_in_decode(gdn, dtype, where):
    c = Case([1] * 3, dtype, 1, 2, 64, 64, seed=2)
    with_top(c, where, 1, 3, 1)
    c.check(decode(gdn, c, c.pool(gdn)))
