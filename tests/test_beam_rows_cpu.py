"""From beam selection to the rows of a fork, by the definitions: a search with
fewer candidates than beams ends rows of its own and touches no other search."""
import numpy as np

import oracle


def rows_of(parents):
    """As the header has it: parent < 0 ? -1 : b * beams + parent."""
    batch, beams = parents.shape
    return np.where(parents < 0, -1, parents + beams * np.arange(batch)[:, None]).reshape(-1)


def test_missing_candidates_end_their_rows():
    rng = np.random.default_rng(0)
    B, W, V, page = 3, 4, 9, 4
    logits = rng.standard_normal((B, W, V))
    logits[1, :, 2:] = -np.inf           # two tokens for each of its two beams with a score
    scores = np.full((B, W), -1.0)
    scores[1, 1:] = -np.inf
    parents = np.stack([oracle.beam_select(logits[b], scores[b], W)[1] for b in range(B)])
    assert (parents[1] == [0, 0, -1, -1]).all() and (parents[[0, 2]] >= 0).all()
    rows = rows_of(parents)
    table = np.arange(B * W * 2).reshape(B * W, 2)
    refs = np.append(np.ones(B * W * 2, dtype=int), np.zeros(9, dtype=int))
    grow = (rows >= 0).astype(int)
    got = oracle.pages_fork(table, np.full(B * W, 6), refs, page, rows, grow, 1)
    assert got["status"] == (0, 0) and (got["lengths"] == np.where(rows < 0, 0, 7)).all()
    assert (got["table"][rows < 0] == -1).all() and (got["slots"][rows < 0] == -1).all()
    # a search's first page is held by its own rows only
    for r, p in enumerate(rows):
        if p >= 0:
            assert p // W == r // W and got["table"][r, 0] == table[p, 0]
    # without the case for -1 the ended rows would be another search's
    wrong = (parents + W * np.arange(B)[:, None]).reshape(-1)
    assert (wrong[rows < 0] // W == 0).all()
