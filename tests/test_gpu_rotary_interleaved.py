"""Rotary positions in place on queries and keys that lie between each other
head by head: the same bits as apart, and the values beside them stay."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


@pytest.mark.parametrize("tokens", [1, 2, 700])
@pytest.mark.parametrize("layout", ["heads inside", "heads outside"])
@pytest.mark.parametrize("adjacent", [False, True])
def test_in_place_between_each_other(tokens, layout, adjacent):
    from activation_sparse_bit_amd import sgemv
    H, D = 6, 80
    g = torch.Generator().manual_seed(tokens)
    shape = (tokens, H, 3, D) if layout == "heads inside" else (H, tokens, 3, D)
    x = torch.randn(*shape, generator=g).half().to(DEV)
    view = x if layout == "heads inside" else x.transpose(0, 1)
    q, k, v = view[:, :, 0], view[:, :, 1], view[:, :, 2]
    positions = torch.randint(0, 9999, (tokens,), generator=g).int().to(DEV)
    inv_freq = (10000.0 ** (-torch.arange(32) / 32.0)).to(DEV)
    pools = lambda: [torch.zeros(-(-tokens // 16), 16, H, D, dtype=torch.float16, device=DEV) for _ in range(2)]  # noqa: E731
    slots = torch.randperm(tokens, generator=g).int().to(DEV)
    apart, kept = [t.contiguous() for t in (q, k, v)], v.clone()
    outs, (k0, v0), (k1, v1) = [torch.empty_like(t) for t in apart[:2]], pools(), pools()
    sgemv.sgemv_rotary(apart[0], outs[0], positions, inv_freq, k=apart[1], k_out=outs[1], v=apart[2],
                       cache=sgemv.KVCache(k0, v0), slots=slots, adjacent=adjacent)
    sgemv.sgemv_rotary(q, q, positions, inv_freq, k=k, k_out=k, v=v, cache=sgemv.KVCache(k1, v1), slots=slots, adjacent=adjacent)
    assert torch.equal(q, outs[0]) and torch.equal(k, outs[1]) and torch.equal(v, kept)
    assert torch.equal(k0, k1) and torch.equal(v0, v1)
