"""The decoding operators at the ends of their ranges: the most heads, tokens
past one launch, caches past 2^32 bytes, the largest vocabulary, a million
pages.  Tolerances as in the operators' own files."""
import numpy as np
import pytest

import oracle
from tests import test_gpu_attention, test_gpu_beam
from tests.test_gpu_pages import Pool

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


def f64(t):
    return t.detach().to(torch.float32).double().cpu().numpy()


@pytest.mark.parametrize("Hq,Hkv,D", [(1024, 1024, 8), (1024, 1, 64), (1024, 512, 16), (1000, 8, 24)])
def test_attention_of_the_most_heads(Hq, Hkv, D):
    test_gpu_attention.Problem(1, [0, 130, 1], Hq, Hkv, D, 16).check()


@pytest.mark.parametrize("heads,dim", [(1024, 256), (1024, 8)])
def test_rotary_of_the_most_heads(heads, dim):
    from activation_sparse_bit_amd import sgemv
    g = torch.Generator().manual_seed(2)
    x = torch.randn(3, heads, dim, generator=g).half()
    inv = 10000.0 ** -(torch.arange(dim // 2) / (dim / 2))
    q, pos = x.to(DEV), torch.tensor([0, 1, 999], dtype=torch.int32)
    sgemv.sgemv_rotary(q, q, pos.to(DEV), inv.to(DEV))
    check_turned(f64(q), f64(x), pos.numpy(), f64(inv))


def check_turned(got, x, positions, inv):
    """Half a step of fp16, and 2^-18 of a pair's length for the roundings in fp32."""
    ref = oracle.rotary(x, positions[None], inv)
    half = x.shape[-1] // 2
    size = np.concatenate([np.hypot(x[..., :half], x[..., half:])] * 2, axis=-1)
    assert (np.abs(got - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -18 * size).all()


def test_rotary_past_one_launch():
    """More tokens than one launch takes, each into its place."""
    from activation_sparse_bit_amd import sgemv
    n = (1 << 22) + 1003
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn(n, 1, 8, generator=g, device=DEV).half() for _ in range(3))
    pages = -(-n // 512)
    kp, vp = (torch.zeros(pages, 512, 1, 8, dtype=torch.float16, device=DEV) for _ in range(2))
    positions = torch.arange(n, dtype=torch.int32, device=DEV) % 5000
    slots = torch.arange(n, dtype=torch.int32, device=DEV).flip(0).contiguous()
    inv = torch.tensor([1.0, 0.1, 0.01, 0.001], device=DEV)
    out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    sgemv.sgemv_rotary(q, out, positions, inv, k=k, k_out=k_out, v=v, cache=sgemv.KVCache(kp, vp), slots=slots)
    for part in (slice(0, 500), slice((1 << 22) - 500, n)):
        for x, got in ((q, out), (k, k_out)):
            check_turned(f64(got[part]), f64(x[part]), positions[part].cpu().numpy(), f64(inv))
    assert torch.equal(kp.view(-1, 1, 8)[:n].flip(0), k_out) and torch.equal(vp.view(-1, 1, 8)[:n].flip(0), v)
    assert int(kp.view(-1, 1, 8)[n:].count_nonzero()) == 0


def test_a_cache_past_32_bits():
    """Writes, copies, forks and compaction behind 2^32 bytes (attention's reads: its own file)."""
    from activation_sparse_bit_amd import sgemv
    pages, page, heads, dim = 40007, 64, 8, 128      # 5.2 GB of keys, as many of values
    kp, vp = (torch.empty(pages, page, heads, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache = sgemv.KVCache(kp, vp)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(3, heads, dim, generator=g).bfloat16().to(DEV) for _ in range(2))
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    last = pages * page - 1
    k_out = torch.empty_like(k)
    sgemv.sgemv_rotary(None, None, i(5, 6, 7), torch.ones(64, device=DEV), k=k, k_out=k_out, v=v, cache=cache,
                       slots=i(last, last - page, last + 1))
    where = ((pages - 1, page - 1), (pages - 2, page - 1))
    for n, (p, t) in enumerate(where):
        assert torch.equal(kp[p, t], k_out[n]) and torch.equal(vp[p, t], v[n])
    sgemv.sgemv_pages_copy([cache], i(pages - 1, 3, page, 5, pages - 3, 10).view(2, 3))
    assert torch.equal(kp[3], kp[pages - 1]) and torch.equal(vp[3], vp[pages - 1]) and torch.equal(vp[pages - 3, :10], vp[5, :10])
    # one row's only page is the last one: a fork copies it, compaction moves it to the front
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[pages - 1] = 1
    refs[:2] = 1                                      # kept by others
    table, lengths = i(pages - 1, -1, -1, -1).view(2, 2), i(page - 5, 0)
    e = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    space = torch.zeros(sgemv.sgemv_pages_workspace_bytes(2, 2, pages), dtype=torch.uint8, device=DEV)
    pairs, count, status = e(2, 3), e(1), e(2)
    sgemv.sgemv_pages_fork(table, lengths, refs, table, lengths, refs, space, page_size=page, parents=i(0, 0), grow=i(1, 1),
                           pairs=pairs, count=count, status=status, caches=[cache])
    assert pairs.tolist()[0] == [pages - 1, 2, page - 5] and count.item() == 1 and status.tolist() == [0, 0]
    assert torch.equal(kp[2, :page - 5], kp[pages - 1, :page - 5])
    refs[2] = 0                                       # (the test's own: its place is free again)
    kept = kp[pages - 1].clone()
    moved = e(pages, 3)
    sgemv.sgemv_pages_compact(table, lengths, refs, table, refs, space, page_size=page, pairs=moved, count=count, caches=[cache])
    assert moved[0].tolist() == [pages - 1, 2, page] and count.item() == 1 and torch.equal(kp[2], kept)
    assert refs[:4].tolist() == [1, 1, 1, 0] and refs[pages - 1].item() == 0


def test_beams_of_the_largest_vocabulary():
    test_gpu_beam.check(*test_gpu_beam.problem(5, 1, 32, 1 << 19, "f16"), 64)
    test_gpu_beam.check(*test_gpu_beam.problem(6, 2, 1, 1 << 19, "f32"), 64)


def test_a_million_pages():
    p = Pool(6, 7, 9, 4, spare=1_100_000, layers=0)
    p.compact()
    p.fork([0, 0, 2, 3, -1, 1, 6], [1, 2, 0, 1, 3, 1, 0])
    p.compact(in_place=True)
