"""Rotary positions, paged attention, beam selection and pages without a GPU:
the oracle against values fixed apart from it, the binding's and the library's
refusals, and the division that places use."""
import math
import random

import numpy as np
import pytest

import oracle
from activation_sparse_bit_amd import sgemv

torch = pytest.importorskip("torch")


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------
def test_rotary_by_complex_numbers():
    rng = np.random.default_rng(1)
    x, pos, f = rng.standard_normal((3, 2, 10)), np.array([[0, 5, -7]]), np.array([1.0, 0.1, 0.03])
    w = np.exp(1j * pos[0][:, None] * f)[:, None]
    got = oracle.rotary(x, pos, f, adjacent=True)
    z = (x[..., 0:6:2] + 1j * x[..., 1:6:2]) * w
    assert np.allclose(got[..., 0:6:2], z.real) and np.allclose(got[..., 1:6:2], z.imag) and (got[..., 6:] == x[..., 6:]).all()
    got = oracle.rotary(x, pos, f, scale=2.0)
    z = (x[..., :3] + 1j * x[..., 3:6]) * w * 2
    assert np.allclose(got[..., :3], z.real) and np.allclose(got[..., 3:6], z.imag)
    # scores depend on the distance only; turning back gives the vector
    q, k = rng.standard_normal((1, 1, 6)), rng.standard_normal((1, 1, 6))
    score = lambda a, b: float((oracle.rotary(q, [[a]], f) * oracle.rotary(k, [[b]], f)).sum())  # noqa: E731
    assert math.isclose(score(3, 8), score(103, 108))
    assert np.allclose(oracle.rotary(oracle.rotary(x, pos, f), -pos, f), x)


def test_rotary_axes():
    assert oracle.rotary_axes([2, 1, 3]) == [0, 0, 1, 2, 2, 2]
    assert oracle.rotary_axes([2, 1, 3], True) == [0, 1, 2, 0, 2, 2]
    assert oracle.rotary_axes([24, 20, 20], True)[:60] == [0, 1, 2] * 20
    x = np.ones((2, 1, 8))
    same = np.array([[4, 9]] * 3)
    assert np.allclose(oracle.rotary(x, same, [1, .5, .2, .1], [1, 2, 1], striped=True), oracle.rotary(x, same[:1], [1, .5, .2, .1]))


def test_attention_by_hand():
    k = np.array([[[1.0, 0]], [[0, 1]], [[1, 1]]])
    v = np.array([[[2.0, 0]], [[0, 4]], [[6, 6]]])
    q = np.array([[math.log(2), 0.0], [0, 0]])
    out, lse, _ = oracle.attention(q, k, v, 1.0)
    assert np.allclose(out[0], [(2 * 2 + 0 + 6 * 2) / 5, (0 + 4 + 12) / 5]) and np.allclose(out[1], [8 / 3, 10 / 3])
    assert np.allclose(lse, [math.log(5), math.log(3)])
    out, lse, _ = oracle.attention(q, k, v, 1.0, window=1)
    assert np.allclose(out, [[6, 6], [6, 6]])
    out, lse, z = oracle.attention(q, k, v, 100.0, softcap=0.5)
    assert np.allclose(z[0], [0.5, 0, 0.5])
    out, lse, _ = oracle.attention(q, k[:0], v[:0], 1.0)
    assert (out == 0).all() and (lse == -np.inf).all()
    # equal keys: the values' mean, whatever the scale; shifting every score shifts lse only
    out, _, _ = oracle.attention(q, np.ones((3, 1, 2)), v, 3.0)
    assert np.allclose(out, v.mean(0))


def test_beam_by_brute_force():
    rng = np.random.default_rng(2)
    for _ in range(20):
        W, V, n = rng.integers(1, 4), rng.integers(1, 6), rng.integers(1, 8)
        logits, scores = rng.integers(-2, 3, (W, V)).astype(float), rng.integers(-3, 1, W).astype(float)
        every = sorted((-(scores[w] + (logits[w, v] - (logits[w].max() + math.log(np.exp(logits[w] - logits[w].max()).sum())))), w, v)
                       for w in range(W) for v in range(V))
        tokens, parents, s, after = oracle.beam_select(logits, scores, n)
        m = min(n, W * V)
        assert np.allclose(s[:m], [-e[0] for e in every[:m]]) and (tokens[m:] == -1).all()
        exact = [(int(w), int(v)) for _, w, v in every[:m]]
        got = list(zip(parents[:m].tolist(), tokens[:m].tolist()))
        if W == 1:
            assert got == [(0, v) for _, v in exact]
    tokens, parents, s, _ = oracle.beam_select([[0.0, 1.0], [5.0, 5.0]], [-1.0, -0.25], 3, [0, 1], 1)
    assert tokens[0] == 1 and parents[0] == 1 and s[0] == -0.25


def test_fork_and_compact_by_hand():
    table = np.array([[3, 5, -1], [3, 6, -1], [9, -1, -1]])
    refs = np.array([0, 0, 0, 2, 0, 1, 1, 0, 0, 1])
    got = oracle.pages_fork(table, [6, 7, 4], refs, 4, parents=[0, 0, -1], grow=[1, 1, 5], max_grow=5)
    # row 2 ends: page 9 is free; row 1 leaves page 6 and shares row 0's page 5, which row 0 copies to 0
    assert got["pairs"].tolist() == [[5, 0, 2], [-1] * 3, [-1] * 3] and got["count"] == 1 and got["status"] == (0, 0)
    assert got["table"].tolist() == [[3, 0, -1], [3, 5, -1], [1, 2, -1]]
    assert got["refs"].tolist() == [1, 1, 1, 2, 0, 1, 0, 0, 0, 0] and got["lengths"].tolist() == [7, 7, 5]
    assert got["slots"].tolist() == [[2, -1, -1, -1, -1], [22, -1, -1, -1, -1], [4, 5, 6, 7, 8]]
    got = oracle.pages_compact(table, [6, 7, 4], refs, 4)
    assert got["pairs"][:4].tolist() == [[5, 0, 4], [6, 1, 4], [9, 2, 4], [-1] * 3] and got["count"] == 3
    assert got["table"].tolist() == [[3, 0, -1], [3, 1, -1], [2, -1, -1]] and got["refs"].tolist() == [1, 1, 1, 2] + [0] * 6


# ---------------------------------------------------------------------------
# the binding's refusals: correct host tensors fail at the device check only
# ---------------------------------------------------------------------------
def cache(pages=4, page=16, heads=2, dim=64, t=torch.float16):
    return sgemv.KVCache(*(torch.zeros(pages, page, heads, dim).to(t) for _ in range(2)))


def refused(call, match):
    with pytest.raises((ValueError, sgemv.SgemvError), match=match):
        call()


def test_cache_refusals():
    z = torch.zeros
    K = sgemv.KVCache
    refused(lambda: K(z(4, 16, 2), z(4, 16, 2)), "k: expected")
    refused(lambda: K(z(4, 16, 2, 64), z(4, 16, 2, 64)), "dtype float32")
    refused(lambda: K(z(4, 16, 2, 64).half(), z(4, 16, 2, 32).half()), "one shape")
    refused(lambda: K(z(4, 16, 2, 64).half(), z(4, 16, 2, 64).bfloat16()), "one shape")
    refused(lambda: K(z(4, 16, 64, 2).half().transpose(2, 3), z(4, 16, 2, 64).half()), "contiguous")
    refused(lambda: K(z(4, 16, 2, 64).half(), z(4, 16, 2, 64).half(), k_scale=z(2)), "k_scale")
    refused(lambda: K(z(4, 16, 2, 64).to(torch.float8_e4m3fn), z(4, 16, 2, 64).to(torch.float8_e4m3fn), v_scale=z(1)), "v_scale")
    refused(lambda: K(np.zeros((4, 16, 2, 64), np.float16), z(4, 16, 2, 64).half()), "k: expected")


def attn(**kw):
    a = {"q": torch.zeros(3, 4, 64).half(), "cache": cache(), "table": torch.zeros(3, 2, dtype=torch.int32),
         "lengths": torch.zeros(3, dtype=torch.int32), "out": torch.zeros(3, 4, 64).half(),
         "workspace": torch.zeros(sgemv.sgemv_attn_workspace_bytes(3, 4, 2, 64), dtype=torch.uint8)}
    a.update(kw)
    return lambda: sgemv.sgemv_attn_paged(**a)


def test_attention_refusals():
    z = torch.zeros
    refused(attn(), "must be a GPU tensor")
    refused(attn(q=z(3, 4, 64)), "float32")
    refused(attn(q=z(3, 256).half()), "q: shape")
    refused(attn(out=z(3, 4, 64).bfloat16()), "out: dtype")
    refused(attn(out=z(2, 4, 64).half()), "out: shape")
    refused(attn(q=z(3, 3, 64).half(), out=z(3, 3, 64).half()), "cache: 2 heads")
    refused(attn(q=z(3, 4, 32).half(), out=z(3, 4, 32).half()), "cache: 2 heads of 64")
    refused(attn(q=z(3, 4, 64).bfloat16(), out=z(3, 4, 64).bfloat16()), "q's type")
    refused(attn(table=z(3, 2)), "table: dtype")
    refused(attn(table=z(2, 2, dtype=torch.int32)), "table: shape")
    refused(attn(table=z(2, 3, dtype=torch.int32).t()), "table: the last")
    refused(attn(lengths=z(4, dtype=torch.int32)), "lengths: shape")
    refused(attn(lengths=z(3, dtype=torch.int64)), "lengths: dtype")
    refused(attn(workspace=z(10)), "workspace")
    refused(attn(lse=z(3, 2)), "lse")
    refused(attn(cache=None), "KVCache")
    refused(attn(window=1 << 40), "window")
    refused(attn(softcap=1e-60), "softcap")
    refused(attn(softcap=-1.0), "softcap")


def rot(**kw):
    a = {"q": torch.zeros(5, 4, 64).half(), "q_out": torch.zeros(5, 4, 64).half(), "positions": torch.zeros(5, dtype=torch.int32),
         "inv_freq": torch.zeros(32), "k": torch.zeros(5, 2, 64).half(), "v": torch.zeros(5, 2, 64).half(), "cache": cache(),
         "slots": torch.zeros(5, dtype=torch.int32)}
    a.update(kw)
    return lambda: sgemv.sgemv_rotary(**a)


def test_rotary_refusals():
    z, i32 = torch.zeros, torch.int32
    refused(rot(), "must be a GPU tensor")
    refused(rot(q_out=None), "both or neither")
    refused(rot(q=z(5, 256).half()), "q: shape")
    refused(rot(q_out=z(5, 4, 64)), "q_out: dtype")
    refused(rot(k=z(4, 2, 64).half()), "k: shape")
    refused(rot(k=None), "cache: needs k")
    refused(rot(cache=None), "k: needs k_out or a cache")
    refused(rot(cache=None, k_out=torch.zeros(5, 2, 64).half()), "v and slots|slots")
    refused(rot(k_out=z(5, 3, 64).half()), "k_out: shape")
    refused(rot(cache=cache(heads=1)), "cache: 1 heads")
    refused(rot(v=z(5, 1, 64).half()), "v: shape")
    refused(rot(slots=z(4, dtype=i32)), "slots: shape")
    refused(rot(slots=None), "slots")
    refused(rot(positions=z(5)), "positions")
    refused(rot(positions=z(3, 4, dtype=i32)), "positions")
    refused(rot(positions=z(5, dtype=i32), sections=[16, 16]), "sections")
    refused(rot(positions=z(2, 5, dtype=i32)), "sections")
    refused(rot(positions=z(2, 5, dtype=i32), sections=[31, 2]), "sections")
    refused(rot(positions=z(2, 5, dtype=i32), sections=[33, -1]), "sections")
    refused(rot(positions=z(5, 5, dtype=i32), sections=[28, 1, 1, 1, 1]), "sections")
    refused(rot(inv_freq=z(32).double()), "inv_freq")


def beam(**kw):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    a = {"logits": torch.zeros(3, 4, 50), "scores": torch.zeros(3, 4), "tokens": i(3, 8), "parents": i(3, 8),
         "scores_out": torch.zeros(3, 8),
         "workspace": torch.zeros(sgemv.sgemv_beam_workspace_bytes(3, 4, 50, 8), dtype=torch.uint8)}
    a.update(kw)
    return lambda: sgemv.sgemv_beam_select(**a)


def test_beam_refusals():
    z = torch.zeros
    refused(beam(), "must be a GPU tensor")
    refused(beam(logits=z(3, 4, 50).double()), "logits: dtype")
    refused(beam(logits=z(3, 200)), "logits: shape")
    refused(beam(scores=z(3, 4).half()), "scores")
    refused(beam(scores=z(4, 4)), "scores")
    refused(beam(tokens=z(3, 8)), "tokens: dtype")
    refused(beam(parents=z(3, 7, dtype=torch.int32)), "parents: shape")
    refused(beam(scores_out=z(24)), "scores_out")
    refused(beam(finished=z(3, 4)), "finished")
    refused(beam(end_token=1 << 31), "end_token")
    refused(beam(workspace=z(3)), "workspace")


def fork(**kw):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    a = {"table": i(4, 6), "lengths": i(4), "refs": i(20), "table_out": i(4, 6), "lengths_out": i(4), "refs_out": i(20),
         "workspace": torch.zeros(sgemv.sgemv_pages_workspace_bytes(4, 6, 20), dtype=torch.uint8), "page_size": 16,
         "pairs": i(4, 3), "count": i(1), "status": i(2), "parents": i(4), "grow": i(4), "slots": i(4, 2)}
    a.update(kw)
    return lambda: sgemv.sgemv_pages_fork(**a)


def test_pages_refusals():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    refused(fork(), "must be a GPU tensor")
    refused(fork(table=i(24)), "table")
    refused(fork(table_out=i(4, 7)), "table_out: 7 columns")
    refused(fork(lengths=i(3)), "lengths: shape")
    refused(fork(refs=i(20).long()), "refs: dtype")
    refused(fork(refs_out=i(19)), "refs_out: shape")
    refused(fork(parents=i(5)), "parents: shape")
    refused(fork(slots=i(8)), "slots")
    refused(fork(slots=i(3, 2)), "slots: shape")
    refused(fork(pairs=i(4, 2)), "pairs: shape")
    refused(fork(status=None), "status")
    refused(fork(caches=[torch.zeros(3)]), "KVCache")
    refused(fork(page_size=1 << 40), "page_size")
    refused(lambda: sgemv.sgemv_pages_copy([cache()], i(3)), "pairs")
    refused(lambda: sgemv.sgemv_pages_copy([], i(3, 3)), "at least one")
    refused(lambda: sgemv.sgemv_pages_copy([cache()], i(3, 3)), "must be a GPU tensor")
    refused(lambda: sgemv.sgemv_pages_copy([cache()] * 129, i(3, 3)), "caches")


# ---------------------------------------------------------------------------
# the library's refusals, before any HIP call (addresses are never followed)
# ---------------------------------------------------------------------------
A = 1 << 40   # an address, and far apart ones


def status(name, packed, *rest):
    return getattr(sgemv.lib(), name)(packed, *rest, 0)


def kv(k=A, v=2 * A, ks=0, vs=0, strides=(2048, 128, 64, 2048, 128, 64), t=0, pages=4, page=16, heads=2, dim=64, reserved=0):
    return sgemv._KV.pack(k, v, ks, vs, *strides, t, pages, page, heads, dim, reserved)


def test_library_refuses_caches():
    def at(**kw):
        args = sgemv._ATTN.pack(3 * A, 4 * A, 0, 5 * A, 6 * A, 7 * A, 1 << 30, 256, 64, 256, 64, 2, kw.pop("type", 0), 1, 4, 2, 0, 1.0, 0.0, 0)
        return status("sgemv_attn_paged", args, kv(**kw))
    assert at(k=0) == at(reserved=1) == at(t=2) == at(t=9) == at(ks=A) == sgemv.SGEMV_EINVAL
    assert at(t=1) == sgemv.SGEMV_EINVAL                                       # neither q's type nor 8 bits
    assert at(pages=0) == at(page=0) == at(page=65537) == at(heads=0) == at(heads=1025) == sgemv.SGEMV_ESIZE
    assert at(dim=0) == at(dim=60) == at(dim=264) == at(pages=1 << 27) == sgemv.SGEMV_ESIZE
    assert at(strides=(2048, 32, 64, 2048, 128, 64)) == at(strides=(2048, 128, 64, -8, 128, 64)) == sgemv.SGEMV_ESIZE
    assert at(k=A + 8) == at(v=2 * A + 2) == at(strides=(2048, 132, 64, 2048, 128, 64)) == sgemv.SGEMV_EALIGN
    assert at(t=3, k=A + 4) == at(t=3, ks=A + 2) == sgemv.SGEMV_EALIGN
    assert at(heads=3, strides=(4096, 256, 64) * 2) == sgemv.SGEMV_EINVAL     # 4 query heads on 3


def test_library_refuses_attention():
    base = dict(q=3 * A, out=4 * A, lse=0, table=5 * A, lengths=6 * A, ws=7 * A, size=1 << 30, q_row=256, q_head=64, out_row=256,
                out_head=64, ld=2, t=0, batch=2, heads=4, pages=2, window=0, scale=1.0, cap=0.0, reserved=0)
    at = lambda **kw: status("sgemv_attn_paged", sgemv._ATTN.pack(*{**base, **kw}.values()), kv())  # noqa: E731
    for kw in (dict(q=0), dict(out=0), dict(table=0), dict(lengths=0), dict(ws=0), dict(t=2), dict(reserved=1), dict(scale=math.inf),
               dict(scale=math.nan), dict(cap=-1.0), dict(cap=math.inf), dict(cap=math.nan), dict(cap=1e-40), dict(heads=5), dict(out=A + 64), dict(out=3 * A + 32),
               dict(lse=4 * A + 4), dict(out=7 * A), dict(lse=A)):
        assert at(**kw) == sgemv.SGEMV_EINVAL, kw
    for kw in (dict(batch=-1), dict(heads=0), dict(heads=2000), dict(pages=0), dict(ld=1), dict(window=-1), dict(size=1000),
               dict(q_head=32), dict(out_row=32), dict(out_row=64), dict(q_row=-64), dict(pages=1 << 27, ld=1 << 27)):
        assert at(**kw) == sgemv.SGEMV_ESIZE, kw
    for kw in (dict(q=3 * A + 1), dict(out=4 * A + 1), dict(lse=8 * A + 2), dict(table=5 * A + 2), dict(lengths=6 * A + 1), dict(ws=7 * A + 128)):
        assert at(**kw) == sgemv.SGEMV_EALIGN, kw
    assert at(batch=0, q=0, out=0) == 0
    L = sgemv.lib()
    assert L.sgemv_attn_paged(None, kv(), 0) == L.sgemv_attn_paged(sgemv._ATTN.pack(*base.values()), None, 0) == sgemv.SGEMV_EINVAL
    for bad in ((-1, 4, 2, 64), (1, 0, 1, 64), (1, 5, 2, 64), (1, 4, 2, 60), (1, 4, 2, 512)):
        assert sgemv.sgemv_attn_workspace_bytes(*bad) == 0
    assert sgemv.sgemv_attn_workspace_bytes(1, 4, 2, 64) > 0


def test_library_refuses_rotary():
    base = dict(q=3 * A, q_out=4 * A, k=5 * A, k_out=0, v=6 * A, pos=7 * A, f=8 * A, slots=9 * A, q_row=256, q_head=64, qo_row=256,
                qo_head=64, k_row=128, k_head=64, ko_row=128, ko_head=64, v_row=128, v_head=64, ld=5, tokens=5, t=0, hq=4, hkv=2,
                dim=64, pairs=32, axes=1, s0=32, s1=0, s2=0, s3=0, flags=0, scale=1.0)
    def at(cache=kv(), **kw):
        return status("sgemv_rotary", sgemv._ROTARY.pack(*{**base, **kw}.values()), cache)
    for kw in (dict(t=3), dict(flags=4), dict(scale=math.nan), dict(s0=31), dict(s0=-1, s1=33, axes=2), dict(s1=1, s0=31), dict(q_out=0),
               dict(q=0), dict(pos=0), dict(f=0), dict(slots=0), dict(k=0), dict(cache=None), dict(cache=kv(dim=32, strides=(1024, 64, 32) * 2)),
               dict(cache=kv(heads=1)), dict(q_out=3 * A + 64), dict(q_out=A + 64), dict(k_out=4 * A), dict(k=A + 16), dict(hq=0)):
        assert at(**kw) == sgemv.SGEMV_EINVAL, kw
    for kw in (dict(tokens=-1), dict(dim=60), dict(dim=512), dict(pairs=0, s0=0), dict(pairs=33, s0=33), dict(axes=0), dict(axes=5),
               dict(q_head=8), dict(qo_row=8), dict(k_row=-1), dict(hq=5000), dict(axes=2, s0=30, s1=2, ld=4), dict(q_row=128)):
        assert at(**kw) == sgemv.SGEMV_ESIZE, kw
    for kw in (dict(q=3 * A + 1), dict(pos=7 * A + 2), dict(f=8 * A + 1), dict(slots=9 * A + 2)):
        assert at(**kw) == sgemv.SGEMV_EALIGN, kw
    assert at(tokens=0) == 0
    assert sgemv.lib().sgemv_rotary(None, None, 0) == sgemv.SGEMV_EINVAL


def test_library_refuses_beams():
    base = dict(logits=A, scores=2 * A, finished=0, tokens=3 * A, parents=4 * A, out=5 * A, ws=6 * A, size=1 << 30, ldb=200, ldw=50, t=2,
                batch=3, beams=4, vocab=50, choices=8, end=0)
    at = lambda **kw: status("sgemv_beam_select", sgemv._BEAM.pack(*{**base, **kw}.values()))  # noqa: E731
    for kw in (dict(logits=0), dict(scores=0), dict(tokens=0), dict(parents=0), dict(out=0), dict(ws=0), dict(t=3), dict(finished=7 * A, end=50),
               dict(finished=7 * A, end=-1), dict(tokens=4 * A + 4), dict(out=A + 8), dict(parents=2 * A), dict(tokens=6 * A)):
        assert at(**kw) == sgemv.SGEMV_EINVAL, kw
    for kw in (dict(batch=-1), dict(beams=0), dict(beams=33), dict(vocab=0), dict(vocab=(1 << 19) + 1), dict(choices=0), dict(choices=65),
               dict(size=100), dict(ldb=-1), dict(ldw=-4)):
        assert at(**kw) == sgemv.SGEMV_ESIZE, kw
    for kw in (dict(logits=A + 2), dict(scores=2 * A + 1), dict(tokens=3 * A + 2), dict(out=5 * A + 2), dict(ws=6 * A + 8)):
        assert at(**kw) == sgemv.SGEMV_EALIGN, kw
    assert at(batch=0, logits=0) == 0
    assert sgemv.sgemv_beam_workspace_bytes(1, 33, 5, 5) == 0
    # a workspace for a batch serves every smaller one
    for beams, vocab, n in ((1, 524288, 1), (4, 32003, 8), (32, 100003, 64), (8, 9000, 16)):
        sizes = [sgemv.sgemv_beam_workspace_bytes(b, beams, vocab, n) for b in (0, 1, 2, 3, 5, 9, 17, 40, 100, 3000)]
        assert sizes == sorted(sizes)


def test_library_refuses_pages():
    base = dict(table=A, lengths=2 * A, refs=3 * A, table_out=4 * A, lengths_out=5 * A, refs_out=6 * A, parents=7 * A, grow=8 * A,
                slots=9 * A, pairs=10 * A, count=11 * A, status=12 * A, ws=13 * A, size=1 << 30, ld=6, ldo=6, rows=4, width=6, pages=20,
                page=16, most=2, layers=0)
    far = kv(k=20 * A, v=21 * A, pages=20)
    def at(name="sgemv_pages_fork", caches=None, **kw):
        return status(name, sgemv._PAGES.pack(*{**base, **kw}.values()), caches)
    for name in ("sgemv_pages_fork", "sgemv_pages_compact"):
        for kw in (dict(table=0), dict(lengths=0), dict(refs=0), dict(table_out=0), dict(refs_out=0), dict(pairs=0), dict(count=0), dict(ws=0),
                   dict(layers=1), dict(table_out=A + 24), dict(refs_out=3 * A + 4), dict(pairs=3 * A), dict(count=13 * A),
                   dict(layers=1, caches=kv(k=A, v=21 * A, pages=20)), dict(layers=1, caches=kv(k=20 * A, v=21 * A, pages=19)),
                   dict(layers=2, caches=far + kv(k=22 * A, v=23 * A, pages=20, t=1))):
            assert at(name, **kw) == sgemv.SGEMV_EINVAL, (name, kw)
        for kw in (dict(rows=0), dict(rows=8193), dict(width=0), dict(pages=0), dict(pages=(1 << 24) + 1), dict(page=0), dict(page=70000),
                   dict(ld=5), dict(ldo=5), dict(size=1000), dict(layers=-1), dict(layers=129)):
            assert at(name, **kw) == sgemv.SGEMV_ESIZE, (name, kw)
        for kw in (dict(table=A + 2), dict(refs_out=6 * A + 1), dict(ws=13 * A + 4)):
            assert at(name, **kw) == sgemv.SGEMV_EALIGN, (name, kw)
    for kw in (dict(lengths_out=0), dict(status=0), dict(lengths_out=8 * A), dict(slots=7 * A), dict(status=10 * A)):
        assert at(**kw) == sgemv.SGEMV_EINVAL, kw
    assert at(most=-1) == at(most=70000) == sgemv.SGEMV_ESIZE and at(grow=8 * A + 2) == sgemv.SGEMV_EALIGN
    L = sgemv.lib()
    assert L.sgemv_pages_copy(far, 1, None, None, 3, 0) == L.sgemv_pages_copy(None, 1, A, None, 3, 0) == sgemv.SGEMV_EINVAL
    assert L.sgemv_pages_copy(far, 0, A, None, 3, 0) == L.sgemv_pages_copy(far, 1, A, None, -1, 0) == sgemv.SGEMV_ESIZE
    assert L.sgemv_pages_copy(far, 1, 20 * A + 64, None, 3, 0) == sgemv.SGEMV_EINVAL
    assert L.sgemv_pages_copy(far, 1, A + 2, None, 3, 0) == sgemv.SGEMV_EALIGN and L.sgemv_pages_copy(far, 1, A, None, 0, 0) == 0


def test_division_by_multiplication():
    """The rule that places use (kv.h): n // d as (n * m) >> s for every n below 2^31 and d up to 65536."""
    rng = random.Random(3)
    for d in list(range(1, 300)) + [2 ** i + j for i in range(9, 17) for j in (-1, 0, 1) if 2 ** i + j <= 65536]:
        s = 31
        while (1 << (s - 31)) < d:
            s += 1
        m = (1 << s) // d + 1
        assert m < 1 << 32
        top = (1 << 31) - 1
        for n in [0, 1, d - 1, d, d + 1, top, top // d * d, top // d * d - 1] + [rng.randrange(1 << 31) for _ in range(20)]:
            assert 0 <= n <= top and (n * m) >> s == n // d or n > top
