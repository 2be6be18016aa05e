"""The bounds that the drafted-tree attention is held to (tests/tree_bounds.py) tell the kernels' formats from coarser ones:
the plain form with its weights rounded as a kernel rounds them keeps its bound, with fewer bits it does not."""
import pytest
import torch

from tests import tree_bounds as T, tree_ref as R


def rounded(x, bits):
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2.0 ** bits) / 2.0 ** bits, e)


@pytest.mark.parametrize("kind,bits,holds", [("bf16", 8, True), ("bf16", 7, False), ("fp8", 11, True), ("fp8", 10, False), ("fp8", 8, False),
                                             ("cores", 24, True), ("cores", 11, False)])
@pytest.mark.parametrize("L", [2, 5, 200])
def test_coarser_weights_leave_the_bound(kind, bits, holds, L):
    if L > 5 and not holds and (kind, bits) != ("fp8", 8):
        return                                                       # many roundings fall against one another
    g = torch.Generator().manual_seed(L)
    worst = 0.0
    for _ in range(40):
        rows = torch.randn(L, 96, generator=g, dtype=torch.float64)
        q = torch.randn(1, 4, 96, generator=g, dtype=torch.float64)
        if L > 5:
            q, rows = 6 * q, rows                                    # one weight far above the others
        see = torch.ones(1, L, dtype=torch.bool)
        o, lse, size, reach = R.attend(q, rows, see, 64, 96 ** -0.5)
        s = q[0] @ rows.T * 96 ** -0.5
        p = torch.exp(s - s.amax(-1, keepdim=True) + 0.3)            # no weight is one
        got = (rounded(p, bits) @ rows[:, :64]) / p.sum(-1, keepdim=True)
        bound = T.o_bound(o, size, reach * 0, 96, L, False, kind)    # the scores are exact here
        worst = max(worst, float(((got - o[0]).abs() / bound[0]).max()))
    assert (worst <= 1) == holds, worst
