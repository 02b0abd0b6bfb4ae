"""Attention of one new token over a paged cache against its float64 definition.

Tolerance.  Products are exact in fp32, so a score is off by its sum's
roundings, at most (dim + 4) * 2^-24 * scale * sum |q k|, and by a few 2^-24 of
its own size when it is scaled and the maximum taken off; with a soft cap, by
the hyperbolic tangent's 4 steps of the cap more.  A probability is off by that
in proportion (called e), by the exponential's 2^-23 and by its rounding to the
inputs' type, half a step (u).  Sums run over at most length / 128 + 64 terms
in a lane and a join, each rounded in fp32, above and below the fraction line.
So out is off by at most (u + 2 e + 4 n 2^-24) * sum p |v| / sum p, plus half a
step of its own type; lse by e + n * 2^-24 and its own rounding."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

T = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
U = 2.0 ** -24
DEV = "cuda:0"


def f64(t):
    return t.detach().to(torch.float32).double().cpu().numpy()


class Problem:
    """A cache whose unused places hold NaN, tables whose unused entries are
    out of range, and the pages of every sequence at random places."""

    def __init__(self, seed, lengths, Hq, Hkv, D, page, x="f16", cache=None, layout="tokens", width=None, scaled=False,
                 poison=True, spread=1.0):
        from activation_sparse_bit_amd import sgemv
        self.lib, cache = sgemv, cache or x
        g = torch.Generator().manual_seed(seed)
        B = len(lengths)
        held = [-(-n // page) for n in lengths]
        pages = sum(held) + 2
        width = width or max(held + [1])
        ids = torch.randperm(pages, generator=g)
        table, at = torch.full((B, width), 1 << 30, dtype=torch.int32), 0
        inner = (Hkv, page, D) if layout == "heads" else (page, Hkv, D)
        pools = []
        for _ in range(2):
            pool = torch.randn(pages, *inner, generator=g) * (spread if cache != "e4m3" else 8.0)
            pools.append(pool.transpose(1, 2) if layout == "heads" else pool)
        mask = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lengths):
            mine = ids[at:at + held[b]]
            table[b, :held[b]] = mine.int()
            at += held[b]
            for i, p in enumerate(mine.tolist()):
                mask[p, :min(page, n - i * page)] = True
        self.pools = []
        for pool in pools:
            if poison:
                pool[~mask] = float("nan")
            self.pools.append(pool.to(T[cache]))
        # copies keep the layout's strides
        self.k, self.v = (p.to(DEV) for p in self.pools)
        self.k, self.v = (torch.empty_strided(p.shape, p.stride(), dtype=p.dtype, device=DEV).copy_(d)
                          for p, d in zip(self.pools, (self.k, self.v)))
        self.scales = [(0.02 + 0.1 * torch.rand(Hkv, generator=g)) if scaled else None for _ in range(2)]
        dev = [None if s is None else s.to(DEV) for s in self.scales]
        self.cache = sgemv.KVCache(self.k, self.v, *dev)
        self.q = torch.randn(B, Hq, D, generator=g).to(T[x])
        self.lengths, self.table = list(lengths), table
        self.dev = [t.to(DEV) for t in (self.q, self.table, torch.tensor(lengths, dtype=torch.int32))]
        self.x, self.Hq, self.Hkv, self.D, self.page = x, Hq, Hkv, D, page
        self.workspace = torch.zeros(sgemv.sgemv_attn_workspace_bytes(B, Hq, Hkv, D), dtype=torch.uint8, device=DEV)

    def run(self, scale=None, window=0, softcap=0.0, out=None, lse=None):
        q, table, lengths = self.dev
        out = torch.full_like(q, 7.0) if out is None else out
        lse = torch.full(q.shape[:2], 7.0, device=DEV) if lse is None else lse
        self.lib.sgemv_attn_paged(q, self.cache, table, lengths, out, self.workspace, scale=scale, window=window,
                                  softcap=softcap, lse=lse)
        return out, lse

    def expected(self, scale=None, window=0, softcap=0.0, only=None):
        scale = self.D ** -0.5 if scale is None else scale
        u, got = torch.finfo(T[self.x]).eps / 2, []
        for b, n in enumerate(self.lengths):
            if only is not None and b not in only:
                got.append(None)
                continue
            pages = self.table[b].tolist()
            k, v = (oracle.paged(f64(p), pages, n) if n else np.zeros((0, self.Hkv, self.D)) for p in self.pools)
            if self.scales[0] is not None:
                k, v = (t * s.double().numpy()[None, :, None] for t, s in zip((k, v), self.scales))
            q = f64(self.q[b])
            out, lse, z = oracle.attention(q, k, v, scale, window, softcap)
            lo = max(0, n - window) if window else 0
            G = self.Hq // self.Hkv
            tol, ltol = np.zeros_like(out), np.zeros(self.Hq)
            for h in range(self.Hq):
                if n == 0:
                    continue
                size = abs(scale) * (np.abs(k[lo:, h // G]) @ np.abs(q[h]))
                top = np.abs(z[h]).max()
                e = ((self.D + 4) * U * size).max() + 8 * U * top + (8 * U * softcap if softcap else 0.0)
                steps = (n - lo) / 128 + 64
                p = np.exp(z[h] - z[h].max())
                weight = p @ np.abs(v[lo:, h // G]) / p.sum()
                tol[h] = (u + 2 * e + 2.0 ** -22 + 4 * steps * U) * weight + np.abs(out[h]) * u + 2.0 ** -24
                ltol[h] = e + 2.0 ** -22 + steps * U + 4 * U * (top + abs(lse[h]))
            got.append((out, tol * 1.01, lse, ltol * 1.01))
        return got

    def check(self, only=None, **kw):
        out, lse = self.run(**kw)
        torch.cuda.synchronize()
        for b, ref in enumerate(self.expected(only=only, **kw)):
            if ref is None:
                continue
            o, tol, l, ltol = ref
            go, gl = f64(out[b]), lse[b].double().cpu().numpy()
            assert np.isfinite(go).all(), (b, "out")
            worst = (np.abs(go - o) - tol).max()
            assert worst <= 0, (b, self.lengths[b], "out", worst, np.abs(go - o).max())
            if self.lengths[b] == 0:
                assert (gl == -np.inf).all() and (go == 0).all()
            else:
                assert (np.abs(gl - l) <= ltol).all(), (b, "lse", np.abs(gl - l).max(), ltol.max())
        assert int(self.workspace[:1 << 18].count_nonzero()) == 0
        return out, lse


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("page", [16, 24])
def test_lengths(n, page):
    Problem(n, [n], 8, 2, 128, page).check()


@pytest.mark.parametrize("D", [8, 24, 56, 64, 72, 80, 96, 112, 120, 128, 136, 160, 192, 200, 224, 256])
@pytest.mark.parametrize("cache", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("page", [32, 5])
def test_head_sizes(D, cache, page):
    x = "f16" if cache == "e4m3" and D % 16 else "bf16" if cache != "f16" else "f16"
    Problem(D, [70, 0, 201], 6, 2, D, page, x, cache, scaled=cache == "e4m3").check()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (4, 4), (12, 4), (16, 1), (17, 1), (33, 1), (40, 2), (71, 1), (64, 8)])
def test_head_counts(Hq, Hkv):
    Problem(Hq, [150, 33], Hq, Hkv, 64, 16, "bf16").check()


@pytest.mark.parametrize("page", [1, 2, 3, 7, 16, 17, 48, 64, 100, 128, 1000])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_pages(page, layout):
    Problem(page, [1, 0, 257, 99], 8, 4, 64, page, layout=layout).check()
    Problem(page, [130], 4, 4, 96, page, "bf16", "e4m3", layout=layout, scaled=True).check()


@pytest.mark.parametrize("window", [1, 2, 16, 31, 100, 128, 129, 400, 5000])
@pytest.mark.parametrize("softcap", [0.0, 2.0, 30.0])
def test_windows_and_soft_caps(window, softcap):
    p = Problem(window, [0, 1, 90, 129, 700], 8, 2, 64, 16, "f16")
    p.check(window=window, softcap=softcap)
    Problem(window, [513, 1], 8, 2, 128, 20, "bf16").check(window=window, softcap=softcap, scale=0.4)


def test_ragged_batches():
    """Lengths from nothing to thousands: runs that hold many sequences, and
    sequences that many runs share."""
    rng = np.random.default_rng(5)
    lengths = [int(n) for n in np.exp(rng.uniform(0, 9, 40))] + [0, 0, 1, 20000]
    Problem(1, lengths, 8, 2, 64, 16).check()
    Problem(2, [0] * 5 + [3] * 300 + [2500], 4, 2, 64, 32, "bf16").check()
    Problem(3, [40000, 1], 4, 1, 64, 64, "bf16").check()


def test_more_sequences_than_a_launch_holds():
    Problem(4, [1 + i % 40 for i in range(2100)], 4, 2, 8, 16).check(only=set(range(0, 2100, 83)) | {2047, 2048, 2099})


def test_large_scores():
    """One token takes all: the others' probabilities vanish without harm."""
    Problem(6, [300, 77], 4, 2, 128, 16, "bf16", spread=8.0).check(scale=1.0)
    Problem(7, [300, 77], 4, 2, 128, 16, "f16", spread=8.0).check(scale=1.0)
    Problem(8, [300], 4, 2, 128, 16, "f16").check(scale=-0.5)
    Problem(9, [300], 4, 2, 128, 16, "f16").check(scale=0.0)


def test_values_that_are_not_finite():
    """Those of seen tokens go through as in the formula, for their head only."""
    p = Problem(10, [200, 200, 200, 200], 8, 4, 64, 16, "f16")
    pages = p.table[:, 3].tolist()
    p.v[pages[0], 2, 0, 5] = float("inf")      # sequence 0, token 50, kv head 0
    p.v[pages[1], 2, 1, 5] = float("nan")
    p.k[pages[2], 2, 2, 5] = float("nan")
    p.dev[0][3, :2] = float("inf")             # scores of infinities and NaN
    out, lse = p.run()
    out, lse = f64(out), lse.cpu().numpy()
    assert (out[0, :2, 5] == np.inf).all() and np.isfinite(np.delete(out[0], 5, axis=1)).all()
    assert np.isnan(out[1, 2:4, 5]).all() and np.isfinite(np.delete(out[1], 5, axis=1)).all()
    assert np.isnan(out[2, 4:6]).all() and np.isnan(lse[2, 4:6]).all() and np.isfinite(out[2, :4]).all()
    assert np.isnan(out[3, :2]).all() and np.isfinite(out[3, 2:]).all()


@pytest.mark.parametrize("page", [16, 24])
def test_bad_pages_and_lengths_make_nan(page):
    """Only the sequences concerned; nothing outside the cache is read."""
    p = Problem(11, [100, 100, 500, 100, 100, 700], 8, 2, 64, page)
    want, _ = p.run()
    table, lengths = p.dev[1].clone(), p.dev[2].clone()
    table[1, 2] = -1
    table[2, 9] = p.cache.pages
    lengths[3] = -5
    lengths[4] = table.shape[1] * page + 1
    out, lse = torch.empty_like(want), torch.empty(6, 8, device=DEV)
    p.lib.sgemv_attn_paged(p.dev[0], p.cache, table, lengths, out, p.workspace, lse=lse)
    for b in range(6):
        if b in (0, 5):
            assert torch.equal(out[b], want[b])
        else:
            assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()


def test_a_long_cache():
    """Places whose byte offsets pass 32 bits: few pages, far apart."""
    from activation_sparse_bit_amd import sgemv
    p = Problem(12, [90, 200], 4, 2, 128, 16, "bf16", poison=False)
    pages, step = p.cache.pages, (5 << 30) // 2 // p.cache.pages // 8 * 8
    far = torch.empty(step * pages, dtype=torch.bfloat16, device=DEV)
    k = far.as_strided(p.k.shape, (step, 256, 128, 1))
    k.copy_(p.k)
    v = torch.as_strided(far, p.v.shape, (step, 256, 128, 1), 16 * 256)
    v.copy_(p.v)
    want = p.run()
    p.cache = sgemv.KVCache(k, v)
    got = p.run()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_strides_and_alignment():
    """Views of wider buffers, at any element; the places around stay as they
    were."""
    p = Problem(13, [60, 140, 9], 6, 2, 40, 16)
    want, want_lse = p.run()
    q0, table0, lengths = p.dev
    for off in (0, 1, 8):
        wide = torch.full((3, 20, 57), 3.0, dtype=torch.float16, device=DEV)
        q, out = wide[:, 1:7, off:off + 40], torch.full((3, 20, 57), 5.0, dtype=torch.float16, device=DEV)
        q.copy_(q0)
        table = torch.full((3, 30), -9, dtype=torch.int32, device=DEV)
        table[:, 2:2 + table0.shape[1]] = table0
        view = out[:, 3:9, off:off + 40]
        p.lib.sgemv_attn_paged(q, p.cache, table[:, 2:2 + table0.shape[1]], lengths, view, p.workspace)
        assert torch.equal(view, want)
        view.fill_(5.0)
        assert (out == 5.0).all()
    # heads outside of rows
    qt, ot = q0.transpose(0, 1).contiguous().transpose(0, 1), torch.empty(6, 3, 40, dtype=torch.float16, device=DEV).transpose(0, 1)
    p.lib.sgemv_attn_paged(qt, p.cache, table0, lengths, ot, p.workspace)
    assert torch.equal(ot, want)


def test_repeats_bit_for_bit_and_in_graphs():
    p = Problem(14, [3000, 0, 17, 9000, 450], 16, 4, 128, 16, "bf16")
    want, want_lse = (t.clone() for t in p.run())
    for _ in range(10):
        out, lse = p.run()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(out=out, lse=lse)
    for n in (3000, 1200, 1, 0, 3000):   # the lengths are read at each replay
        p.dev[2][0] = n
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = p.run()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
    assert torch.equal(out, want)


def test_one_workspace_serves_other_shapes_and_streams():
    a = Problem(15, [500, 900], 8, 2, 128, 16)
    b = Problem(16, [70] * 9, 4, 4, 64, 24, "bf16")
    want_a, want_b = a.run()[0].clone(), b.run()[0].clone()
    b.workspace = a.workspace
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(3):
            assert torch.equal(a.run()[0], want_a)
            assert torch.equal(b.run()[0], want_b)
    stream.synchronize()


def test_empty_batch():
    p = Problem(17, [5], 4, 2, 64, 16)
    e = lambda *s, t=torch.int32: torch.empty(*s, dtype=t, device=DEV)  # noqa: E731
    p.lib.sgemv_attn_paged(e(0, 4, 64, t=torch.float16), p.cache, e(0, 3), e(0), e(0, 4, 64, t=torch.float16), p.workspace)
    torch.cuda.synchronize()
