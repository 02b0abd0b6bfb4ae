"""Rotary positions and the write into a paged cache against the float64
definition.

Tolerance.  The part of a turn that an angle leaves is formed in 64 bits (off
by 2^-52 of the turns) and rounded to fp32, at most 2^-25 of a turn; cosine and
sine of it are off by two steps of 2^-23 more: in all at most 2 pi (2^-25 +
2^-52 turns) + 2^-22.  A turned value adds three roundings of 2^-24 of
|a| + |b|, and half a step of its type; in an 8-bit cache half a step of that
(2^-4 of the value, 2^-10 below 2^-6) after a division by the scale."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150, "e4m3": 2.0 ** -10}
DEV = "cuda:0"


def f64(t):
    return t.detach().to(torch.float32).double().cpu().numpy()


def half_step(v, t):
    return np.abs(v) * torch.finfo(T[t]).eps / 2 + TINY[t]


def tolerance(x, positions, inv_freq, scale):
    """Before the last rounding, for every value of a [tokens][heads][dim]."""
    turns = np.abs(positions).max() * float(inv_freq.max()) / (2 * np.pi)
    e = 2 * np.pi * (2.0 ** -25 + 2.0 ** -52 * (turns + 1)) + 2.0 ** -22 + 4 * 2.0 ** -24
    return abs(scale) * e * 2 * np.abs(x).max(-1, keepdims=True) * np.ones_like(x)


def check(seed, tokens, Hq, Hkv, D, pairs, x="f16", sections=None, axes=1, adjacent=False, striped=False, scale=1.0,
          cache=None, page=16, layout="tokens", far=4000, scaled=False, pad=0, in_place=False, with_k_out=True):
    from activation_sparse_bit_amd import sgemv
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(tokens, Hq + 2 * Hkv, D + pad, generator=g).to(T[x]).to(DEV)[:, :, pad:]
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    kept = [t.clone() for t in (q, k, v)]
    positions = torch.randint(-far, far + 1, (axes, tokens), generator=g).int()
    inv_freq = (10000.0 ** (-torch.arange(pairs).double() / pairs)).float()
    q_out, k_out = (q, k) if in_place else (torch.full_like(q.contiguous(), 9.0), torch.full_like(k.contiguous(), 9.0))
    kw, pools, scales, slots = {}, None, (None, None), None
    if cache:
        pages = -(-tokens // page) + 2
        inner = (Hkv, page, D) if layout == "heads" else (page, Hkv, D)
        pools = [torch.full((pages, *inner), 3.0).to(T[cache]).to(DEV) for _ in range(2)]
        pools = [p.transpose(1, 2) if layout == "heads" else p for p in pools]
        if scaled:
            scales = tuple((0.005 + 0.05 * torch.rand(Hkv, generator=g)).to(DEV) for _ in range(2))
        slots = torch.randperm(pages * page, generator=g)[:tokens].int()
        if tokens > 3:
            slots[1], slots[2] = -1, pages * page   # not written
        kw = {"v": v, "cache": sgemv.KVCache(*pools, *scales), "slots": slots.to(DEV)}
    pos = positions.to(DEV) if axes > 1 else positions[0].to(DEV)
    sgemv.sgemv_rotary(q, q_out, pos, inv_freq.to(DEV), k=k, k_out=k_out if with_k_out or not cache else None,
                       sections=sections, adjacent=adjacent, striped=striped, scale=scale, **kw)
    torch.cuda.synchronize()
    refs = []
    for t, out in ((kept[0], q_out), (kept[1], k_out)):
        ref = oracle.rotary(f64(t), positions.numpy(), inv_freq.numpy(), sections, adjacent, striped, scale)
        tol = tolerance(f64(t), positions.numpy(), inv_freq.numpy(), scale)
        refs.append((ref, tol))
        if out is q_out or with_k_out or not cache:
            over = np.abs(f64(out) - ref) - (tol + half_step(ref, x)) * 1.01
            assert (over <= 0).all(), over.max()
            assert (f64(out)[..., 2 * pairs:] == f64(t)[..., 2 * pairs:]).all()
        else:
            assert (out == 9.0).all()
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip((q, k, v), kept))
    if cache:
        written = [(t, s) for t, s in enumerate(slots.tolist()) if 0 <= s < pages * page]
        for pool, (ref, tol), scl in zip(pools, (refs[1], (f64(kept[2]), np.zeros(kept[2].shape))), scales):
            got, rest = f64(pool), np.ones((pages, page), dtype=bool)
            by = 1.0 if scl is None else f64(scl)[:, None]
            for t, s in written:
                want, err = ref[t] / by, tol[t] / by
                if cache == "e4m3":
                    want = np.clip(want, -448, 448)
                over = np.abs(got[s // page, s % page] - want) - (err + 2.0 ** -23 * np.abs(want) + half_step(want, cache)) * 1.01
                assert (over <= 0).all(), (t, s, over.max())
                rest[s // page, s % page] = False
            assert (got[rest] == 3.0).all()


@pytest.mark.parametrize("D,pairs", [(8, 4), (8, 1), (64, 32), (72, 36), (80, 40), (96, 24), (96, 48), (104, 5), (128, 64),
                                     (128, 16), (200, 100), (256, 128), (256, 120)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("x", ["f16", "bf16", "f32"])
def test_head_sizes(D, pairs, adjacent, x):
    check(D + pairs, 5, 6, 2, D, pairs, x, adjacent=adjacent, cache="bf16" if x == "bf16" else "f16")


@pytest.mark.parametrize("axes,sections", [(1, [16]), (2, [10, 6]), (3, [6, 5, 5]), (3, [0, 16, 0]), (4, [1, 2, 3, 10])])
@pytest.mark.parametrize("striped", [False, True])
@pytest.mark.parametrize("adjacent", [False, True])
def test_axes(axes, sections, striped, adjacent):
    check(axes, 33, 4, 2, 40, 16, "f32", sections, axes, adjacent, striped)


@pytest.mark.parametrize("cache", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
@pytest.mark.parametrize("x", ["f16", "f32"])
def test_caches(cache, page, layout, x):
    check(page, 40, 4, 2, 64, 32, x, cache=cache, page=page, layout=layout, scaled=cache == "e4m3", with_k_out=page != 7)
    check(page + 1, 3, 1, 3, 24, 5, x, cache=cache, page=page, layout=layout, scale=0.7)


@pytest.mark.parametrize("tokens", [1, 2, 3, 31, 500, 513, 3001])
def test_token_counts(tokens):
    check(tokens, tokens, 8, 2, 64, 32, "bf16", cache="bf16")
    check(tokens, tokens, 3, 1, 16, 8, "f16", in_place=True)


@pytest.mark.parametrize("far", [1, 1 << 20, (1 << 31) - 2])
def test_far_positions(far):
    check(3, 50, 2, 1, 128, 64, "f32", far=far)


@pytest.mark.parametrize("pad", [0, 1, 4, 8])
@pytest.mark.parametrize("x", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
def test_alignment_and_in_place(pad, x, adjacent):
    check(pad, 9, 4, 2, 64, 24, x, adjacent=adjacent, pad=pad, cache="f16", in_place=pad % 2 == 0)


def test_queries_or_keys_alone():
    from activation_sparse_bit_amd import sgemv
    q = torch.randn(4, 3, 16, device=DEV)
    pos, f = torch.arange(4, dtype=torch.int32, device=DEV), torch.ones(8, device=DEV)
    a, b = torch.empty_like(q), torch.empty_like(q)
    sgemv.sgemv_rotary(q, a, pos, f)
    sgemv.sgemv_rotary(None, None, pos, f, k=q, k_out=b)
    assert torch.equal(a, b)
    none = q[:0]
    sgemv.sgemv_rotary(none, a[:0], pos[:0], f)


def test_saturation_and_nan_in_8_bits():
    from activation_sparse_bit_amd import sgemv
    k = torch.zeros(1, 1, 8, device=DEV)
    v = torch.tensor([[[1e6, -1e6, 448.0, 470.0, float("nan"), float("inf"), -float("inf"), 0.001]]], device=DEV)
    pools = [torch.zeros(1, 1, 1, 8, device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
    sgemv.sgemv_rotary(None, None, torch.zeros(1, dtype=torch.int32, device=DEV), torch.ones(1, device=DEV), k=k, v=v,
                       cache=sgemv.KVCache(*pools), slots=torch.zeros(1, dtype=torch.int32, device=DEV))
    got = pools[1].float().flatten().tolist()
    assert got[:4] == [448.0, -448.0, 448.0, 448.0] and got[4] != got[4] and got[5:7] == [448.0, -448.0]
    assert abs(got[7] - 0.001) <= 2.0 ** -10


def test_graph():
    from activation_sparse_bit_amd import sgemv
    q = torch.randn(6, 4, 64, device=DEV).half()
    pools = [torch.zeros(2, 16, 4, 64, device=DEV).half() for _ in range(2)]
    cache = sgemv.KVCache(*pools)
    pos, slots = torch.arange(6, dtype=torch.int32, device=DEV), torch.arange(6, dtype=torch.int32, device=DEV)
    f, out = torch.rand(32, device=DEV), torch.empty_like(q)
    run = lambda o: sgemv.sgemv_rotary(q, o, pos, f, k=q, v=q, cache=cache, slots=slots)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    run(out)
    with torch.cuda.graph(graph):
        run(out)
    for i in range(4):
        pos += 100 * i
        slots += i
        graph.replay()
        got, k = out.clone(), pools[0].clone()
        run(out)
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(pools[0], k)
