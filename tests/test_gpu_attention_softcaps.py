"""Soft caps of every size: softcap * tanh(z / softcap) is z itself under a cap
far above all scores, up to the largest float, and the cap's sign under one far
below them, down to the smallest normal float.

Tolerance.  As without a cap (test_gpu_attention), with 8 * 2^-24 of the largest
score more for the tangent, and with 2^-22 for caps above 2^126, whose
reciprocal is off by 2^-150 and so a score by 2^-150 times the cap at most."""
import numpy as np
import pytest

from tests import test_gpu_attention as base

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U, f64 = 2.0 ** -24, base.f64
LARGEST = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("cap", [1e4, 1e30, 2.0 ** 126, 2.3e38, 2.4e38, 3e38, LARGEST])
@pytest.mark.parametrize("x", ["f16", "bf16"])
def test_caps_far_above_the_scores(cap, x):
    p = base.Problem(31, [1, 33, 700, 0], 8, 2, 64, 16, x)
    p.k[p.table[1, 0], 3] = 0   # scores of zero among them
    p.pools[0] = p.k.cpu()
    out, lse = p.run(softcap=cap)
    for b, ref in enumerate(p.expected(softcap=0.0)):
        o, tol, l, ltol = ref
        # z - cap tanh(z / cap) is z^3 / (3 cap^2) at most: 2e-6 at a cap of 1e4 and scores of 8
        more = 8 * U * 8 + 2.0 ** -22 + 8.0 ** 3 / (3 * min(cap, 1e18) ** 2)
        assert (np.abs(f64(out[b]) - o) <= tol + 2 * more * 4).all(), (b, np.abs(f64(out[b]) - o).max())
        got = lse[b].double().cpu().numpy()
        with np.errstate(invalid="ignore"):   # -infinity less itself, for the empty sequence
            assert ((got == l) | (np.abs(got - l) <= ltol + more)).all(), (b, got, l)


@pytest.mark.parametrize("cap", [float(np.finfo(np.float32).tiny), 1e-30, 1e-10])
def test_caps_far_below_the_scores(cap):
    """All probabilities are equal, within the cap: the values' mean, scores of zero among them."""
    p = base.Problem(32, [1, 33, 700, 0], 8, 2, 64, 16)
    p.k[p.table[1, 0], 3] = 0
    p.pools[0] = p.k.cpu()
    p.check(softcap=cap)


def test_infinite_scores_are_capped():
    """Queries whose scores overflow have the cap as their score."""
    p = base.Problem(33, [200], 4, 2, 64, 16, "bf16")
    p.dev[0].fill_(3e38)
    p.k.copy_(torch.where(torch.isnan(p.k), p.k, torch.ones_like(p.k)))
    out, lse = p.run(softcap=5.0)
    assert torch.isfinite(out).all() and (lse.double() - 5.0 - np.log(200.0)).abs().max() < 1e-5
