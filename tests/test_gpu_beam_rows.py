"""Beam selection and the fork that follows it, where a search has fewer
candidates than beams: its missing rows end, and the other searches' pages,
counts and rows are as if it were not there."""
import pytest

import oracle
from tests import test_gpu_beam, test_gpu_pages

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


@pytest.mark.parametrize("B,W", [(2, 4), (5, 3)])
def test_missing_candidates_end_their_rows(B, W):
    V = 1003
    logits, scores = test_gpu_beam.problem(B, B, W, V, "f32")
    short = B - 1                       # the last search: one beam, two tokens
    scores[short, 1:] = -float("inf")
    logits[short, 0, 2:] = -float("inf")
    test_gpu_beam.check(logits, scores, W)
    tokens, from_beam, _ = test_gpu_beam.run(logits, scores, W)
    assert (from_beam[short, 2:] == -1).all() and (from_beam[:short] >= 0).all()
    first_row = W * torch.arange(B, device=DEV, dtype=torch.int32)
    parents = torch.where(from_beam < 0, -1, from_beam + first_row[:, None]).view(-1).tolist()
    p = test_gpu_pages.Pool(B, B * W, 6, 4)
    before = p.table.copy(), p.lengths.copy(), p.refs.copy()
    grow = [int(x >= 0) for x in parents]
    p.fork(parents, grow)               # checked against the definition, copies with it
    # the pages that the other searches go on with are counted as if the short one ended whole
    table, lengths, refs = before
    rest = [x if r < short * W else -1 for r, x in enumerate(parents)]
    alone = oracle.pages_fork(table, lengths, refs, 4, rest, [g if r < short * W else 0 for r, g in enumerate(grow)], 1)
    held = lambda r: set(table[r, :-(-int(lengths[r]) // 4)].tolist())  # noqa: E731
    mine = set().union(*(held(x) for x in rest[:short * W])) - set().union(*(held(r) for r in range(short * W, B * W)))
    assert mine and all(p.refs[i] == alone["refs"][i] for i in mine)
    ended = [r for r, x in enumerate(parents) if x < 0]
    assert ended and (p.lengths[ended] == 0).all() and (p.table[ended] == -1).all()
