"""Beam selection against its float64 definition.

Tolerance.  A sum of exponentials in fp32 has at most 32 terms a thread, 6 steps
over a wavefront and 3 over the wavefronts, each off by 2^-24, the exponentials
by 2^-22; the parts are joined in 64 bits.  Its logarithm, and so a score, is
off by at most 64 * 2^-24, and by half a step of fp32 when it is written.
Tokens and parents are the definition's wherever two scores of different beams
are further apart than twice that; scores of one beam are ordered exactly."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"
E = 64 * 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def run(logits, scores, n, finished=None, end=0, workspace=None, out=None):
    from activation_sparse_bit_amd import sgemv
    B, W, V = logits.shape
    if out is None:
        out = (torch.full((B, n), 77, dtype=torch.int32, device=DEV), torch.full((B, n), 77, dtype=torch.int32, device=DEV),
               torch.full((B, n), 77.0, device=DEV))
    if workspace is None:
        workspace = torch.zeros(sgemv.sgemv_beam_workspace_bytes(B, W, V, n), dtype=torch.uint8, device=DEV)
    sgemv.sgemv_beam_select(logits, scores, *out, workspace, finished=finished, end_token=end)
    assert int(workspace[:1 << 17].count_nonzero()) == 0
    return out


def check(logits, scores, n, finished=None, end=0, exact=False):
    tokens, parents, got = run(logits, scores, n, finished, end)
    for b in range(logits.shape[0]):
        rt, rp, rs, after = oracle.beam_select(f64(logits[b]), f64(scores[b]), n,
                                               None if finished is None else finished[b].tolist(), end)
        gt, gp, gs = tokens[b].cpu().numpy(), parents[b].cpu().numpy(), f64(got[b])
        there = np.isfinite(rs)
        assert (gt[~there] == -1).all() and (gp[~there] == -1).all() and (gs[~there] == -np.inf).all()
        tol = E + np.abs(rs[there]) * 2.0 ** -23 + E
        assert (np.abs(gs[there] - rs[there]) <= tol).all(), np.abs(gs[there] - rs[there]).max()
        # a place is certain where its neighbours are of the same beam or far enough away
        with np.errstate(invalid="ignore"):
            near = np.abs(np.diff(np.append(rs, after))) <= 2 * E
        beam = np.append(rp, -2)
        doubt = near & (beam[1:] != beam[:-1])
        if exact:
            doubt[:] = False
        sure = there & ~(doubt | np.append(False, doubt[:-1]))
        assert (gt[sure] == rt[sure]).all() and (gp[sure] == rp[sure]).all(), (b, gt, rt, gp, rp)
        assert sure.sum() >= there.sum() - 4 or not there.any()


def problem(seed, B, W, V, x, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(B, W, V, generator=g)).to(T[x]).to(DEV), (-9 * torch.rand(B, W, generator=g)).to(DEV)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 255, 2047, 2048, 2049, 8192, 8193, 20001])
@pytest.mark.parametrize("x", ["f16", "bf16", "f32"])
def test_vocabularies(V, x):
    check(*problem(V, 3, 4, V, x), 8)


@pytest.mark.parametrize("W,n", [(1, 1), (1, 64), (2, 4), (5, 3), (8, 16), (16, 32), (32, 64), (31, 63)])
def test_beams_and_choices(W, n):
    check(*problem(W, 2, W, 3001, "f32"), n)
    check(*problem(W, 1, W, 5, "bf16"), n)


@pytest.mark.parametrize("B", [1, 7, 200])
def test_batches(B):
    check(*problem(B, B, 4, 900, "bf16"), 8)


def test_large_vocabulary_and_the_coarse_cut():
    check(*problem(1, 1, 2, 1 << 19, "bf16"), 16)
    check(*problem(2, 40, 8, 16500, "f16"), 16)
    check(*problem(3, 40, 8, 16500, "f32"), 64)
    check(*problem(4, 1, 32, 1 << 18, "f32"), 64)
    check(*problem(5, 1, 8, 100003, "bf16"), 16)
    check(*problem(6, 1, 3, 40000, "f16"), 6)


def test_more_entries_than_a_launch_holds():
    logits, scores = problem(4, 2100, 2, 50, "f32")
    check(logits, scores, 4)


def test_ties_go_to_the_lowest_place():
    """Equal logits, sorted logits, equal beams: every value is a candidate's
    equal, or many values are near the bound."""
    for x in T:
        flat = torch.zeros(1, 3, 9000, device=DEV).to(T[x])
        check(flat, torch.zeros(1, 3, device=DEV), 16, exact=True)
        check(flat - 2.5, torch.tensor([[0.0, 1.0, 1.0]], device=DEV), 64, exact=True)
    up = torch.arange(9000, device=DEV).float()[None, None] / 9000
    check(up.repeat(1, 2, 1), torch.zeros(1, 2, device=DEV), 64, exact=True)
    check(up.flip(-1).repeat(1, 2, 1).contiguous(), torch.zeros(1, 2, device=DEV), 64, exact=True)
    check(up.repeat(1, 2, 1).bfloat16(), torch.zeros(1, 2, device=DEV), 33, exact=True)
    zeros = torch.zeros(1, 1, 4000, device=DEV)
    zeros[0, 0, ::2] = -0.0   # minus zero is zero
    check(zeros, torch.zeros(1, 1, device=DEV), 7, exact=True)
    few = torch.randint(-3, 3, (2, 4, 30000), device=DEV).float()
    check(few.half(), torch.zeros(2, 4, device=DEV), 20, exact=True)


def test_forbidden_tokens_and_beams_without_candidates():
    logits, scores = problem(5, 6, 4, 3000, "f32")
    logits[0, :, 10:] = -float("inf")        # ten tokens each
    logits[1, 1:] = -float("inf")            # one beam
    logits[2] = -float("inf")                # none
    logits[3, 0, 5] = float("nan")           # not a candidate
    logits[4, 2, 7] = float("inf")           # no normaliser: beam 2 has none
    scores[5] = torch.tensor([-1.0, -float("inf"), float("nan"), float("inf")])
    logits[0, 2] = -float("inf")
    check(logits, scores, 32)
    tokens, parents, got = run(logits, scores, 32)
    assert (tokens[2] == -1).all() and (parents[1] == 0).all() and (parents[5] == 0).all() and not (parents[4] == 2).any()
    assert int((tokens[0] >= 0).sum()) == 30


def test_finished_beams():
    logits, scores = problem(6, 5, 4, 700, "bf16")
    finished = torch.zeros(5, 4, dtype=torch.uint8, device=DEV)
    finished[1, 2] = finished[2] = 1
    finished[3, :3] = 1
    scores[3, 1] = -float("inf")
    logits[2] = float("nan")                 # never read
    check(logits, scores, 8, finished, end=699)
    check(logits, scores, 8, finished.bool(), end=0)
    tokens, parents, got = run(logits, scores, 8, finished, 11)
    assert sorted(parents[2, :4].tolist()) == [0, 1, 2, 3] and (tokens[2, :4] == 11).all() and (tokens[2, 4:] == -1).all()


def test_strides_and_alignment():
    logits, scores = problem(7, 3, 4, 1001, "f16")
    want = run(logits, scores, 8)
    for off in (0, 1, 3):
        wide = torch.full((3, 6, 1013), float("inf"), dtype=torch.float16, device=DEV)
        view = wide[:, 1:5, off:off + 1001]
        view.copy_(logits)
        for a, b in zip(want, run(view, scores, 8)):
            assert torch.equal(a, b)
    turned = logits.transpose(0, 1).contiguous().transpose(0, 1)
    for a, b in zip(want, run(turned, scores, 8)):
        assert torch.equal(a, b)


def test_repeats_graph_and_shared_workspace():
    from activation_sparse_bit_amd import sgemv
    a, b = problem(8, 4, 8, 30000, "bf16"), problem(9, 1, 3, 999, "f32")
    space = torch.zeros(max(sgemv.sgemv_beam_workspace_bytes(4, 8, 30000, 16), sgemv.sgemv_beam_workspace_bytes(1, 3, 999, 6)),
                        dtype=torch.uint8, device=DEV)
    want_a, want_b = run(*a, 16, workspace=space), run(*b, 6, workspace=space)
    out = tuple(torch.zeros_like(t) for t in want_a)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sgemv.sgemv_beam_select(*a, *out, space)
    for _ in range(5):
        for t in out:
            t.zero_()
        graph.replay()
        for x, y in zip(want_b, run(*b, 6, workspace=space)):
            assert torch.equal(x, y)
        for x, y in zip(want_a, out):
            assert torch.equal(x, y)


@pytest.mark.parametrize("fill", [-1e9, -1e10, -1e30, "lowest", 1e9, 1e30, "half of the largest"])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_logits_far_from_zero(fill, x):
    """Beams, and whole parts of a vocabulary, that hold one value far from zero, as masks leave them."""
    big = torch.finfo(T[x]).max
    fill = {"lowest": -big, "half of the largest": big / 2}.get(fill, fill)
    _, scores = problem(10, 3, 4, 1, x)
    logits = torch.full((3, 4, 30001), fill, device=DEV).to(T[x])
    check(logits, scores, 9)                                     # every beam even
    some = logits.clone()
    g = torch.Generator().manual_seed(11)
    some[:, :, ::4001] = torch.randn(3, 4, 8, generator=g).to(T[x]).to(DEV)
    check(some, scores, 9)                                       # few others, here and there
    some[:, 2:] = logits[:, 2:]
    some[0, 1, 100:200] = float("-inf")
    some[1, 2, 5] = float("nan")
    some[1, 3, 29000:] = -big
    check(some, scores, 40)
