"""Beam selection where many values are equal: parts that keep more values than
are ranked at once, and entries with more than 2 n + 96 candidates at the end,
for every number of runs that a thread takes.  Both ways go through the step
that drops candidates, whose count all threads have to agree on."""
import pytest

from tests import test_gpu_beam as base

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# beams and vocabulary so that a thread has one, two and four runs of eight
CUTS = [(1, 2, 30000), (2, 16, 40000), (1, 32, 70000)]


@pytest.mark.parametrize("B,W,V", CUTS)
@pytest.mark.parametrize("n", [2, 16, 17, 64])
@pytest.mark.parametrize("x", ["f16", "bf16", "f32"])
def test_flat_logits(B, W, V, n, x):
    """Everything is equal: the answer is the first tokens of the first beam."""
    flat = torch.full((B, W, V), -1.5, device=base.DEV).to(base.T[x])
    tokens, parents, scores = base.run(flat, torch.zeros(B, W, device=base.DEV), n)
    assert (tokens == torch.arange(n, device=base.DEV, dtype=torch.int32)).all() and (parents == 0).all()
    assert (scores == scores[0, 0]).all()


@pytest.mark.parametrize("B,W,V", CUTS)
@pytest.mark.parametrize("n", [16, 33, 64])
def test_few_values(B, W, V, n):
    """Some values, each a thousand times; beams with the same values, so that candidates of all of them compete."""
    g = torch.Generator().manual_seed(V + n)
    row = torch.randint(-4, 5, (V,), generator=g).float()
    logits = torch.stack([row.roll(7 * w) for w in range(W)])[None].repeat(B, 1, 1).half().to(base.DEV)
    # beams' scores apart from each other: equal sums are rounded in another order in another beam
    base.check(logits, (-0.01 * torch.arange(W).float())[None].repeat(B, 1).to(base.DEV), n)


@pytest.mark.parametrize("n", [16, 64])
def test_repeats(n):
    """Many entries, so that the GPU is full while the last workgroups choose: the same bits every time."""
    flat = torch.zeros(64, 4, 20000, device=base.DEV).bfloat16()
    flat[:, :, ::3] = 1.0
    scores = torch.zeros(64, 4, device=base.DEV)
    want = [t.clone() for t in base.run(flat, scores, n)]
    assert (want[0] == 3 * torch.arange(n, device=base.DEV, dtype=torch.int32)).all() and (want[1] == 0).all()
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(want, base.run(flat, scores, n)))
