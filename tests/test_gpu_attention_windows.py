"""Attention with a window over pages that were given back: table entries whose
tokens all lie before the window are not in use, whatever stands there."""
import pytest

from tests import test_gpu_attention as base

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def give_back(p, window, with_):
    """Replaces, on the device, every entry that no seen token is in."""
    table = p.table.clone()
    for b, n in enumerate(p.lengths):
        table[b, :max(0, n - window) // p.page] = with_
    p.dev[1].copy_(table.to(base.DEV))


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 32, 48])
@pytest.mark.parametrize("window", [1, 5, 100, 128])
def test_entries_before_a_window_are_not_in_use(page, window):
    """Lengths of every remainder, so that the window begins everywhere in a step of 32 tokens."""
    p = base.Problem(page + window, list(range(170, 234)) + [1, 0, window], 4, 2, 64, page, "bf16")
    want = p.check(window=window)
    for with_ in (-1, 1 << 30, p.cache.pages):
        give_back(p, window, with_)
        got = p.run(window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("page,D,cache", [(8, 128, "f16"), (16, 128, "e4m3"), (64, 256, "f16"), (24, 96, "e4m3")])
def test_long_sequences_with_a_window(page, D, cache):
    """Windows that many workgroups share, beside short ones; entries in use still make NaN where they are no pages."""
    p = base.Problem(page, [30000, 5003, 2500, 17, 9001], 8, 2, D, page, "f16", cache)
    want = p.check(window=4100)
    give_back(p, 4100, -1)
    got = p.run(window=4100)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    p.dev[1][0, (30000 - 4100) // page] = -1   # the first entry of the window
    out, lse = p.run(window=4100)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all() and torch.equal(out[1:], want[0][1:])
