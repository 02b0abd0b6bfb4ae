"""The 4-bit products and the block norm without a GPU: the packer byte for
byte against the layout formula, the header round trip, the oracle against
closed forms and exact rationals, and every refusal before any HIP call."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import oracle
from activation_sparse_bit_amd import sgemv

E = sgemv
FAKE = 1 << 20   # a well-aligned address that no call here dereferences


def problem(seed, N, K, group, zeros=True):
    rng = np.random.default_rng(seed)
    G = -(-K // group)
    q = rng.integers(0, 16, (N, K), dtype=np.uint8)
    s = rng.uniform(0.003, 0.02, (N, G)).astype(np.float16)
    z = rng.integers(0, 16, (N, G), dtype=np.uint8) if zeros else None
    return q, s, z


def bits(s):
    return s.view(np.uint16)


@pytest.mark.parametrize("N,K,group", [(1, 1, 128), (16, 128, 128), (17, 129, 32), (33, 257, 64), (5, 31, 32),
                                       (48, 640, 128), (31, 96, 64)])
@pytest.mark.parametrize("zeros", [True, False])
def test_packer_matches_formula(N, K, group, zeros):
    q, s, z = problem(N * 31 + K, N, K, group, zeros)
    d, blob = sgemv.sgemv_q4_pack(q, s, z, group)
    ref = oracle.q4_pack_spec([(q, bits(s), z)], group)
    assert blob.shape == ref.shape and np.array_equal(blob, ref)
    flags = sgemv.SGEMV_Q4_ZEROS if zeros else 0
    assert d.as_dict() == oracle.q4_header_fields(N, K, group, flags)
    assert sgemv.sgemv_q4_desc_from_header(blob).as_dict() == d.as_dict()


@pytest.mark.parametrize("N,K,group", [(1, 1, 32), (16, 128, 64), (19, 300, 128)])
def test_gated_packer_matches_formula(N, K, group):
    gate, up = problem(1, N, K, group), problem(2, N, K, group)
    d, blob = sgemv.sgemv_q4_pack_gated(gate, up, group)
    ref = oracle.q4_pack_spec([(p[0], bits(p[1]), p[2]) for p in (gate, up)], group)
    assert np.array_equal(blob, ref)
    assert d.flags == sgemv.SGEMV_Q4_GATED | sgemv.SGEMV_Q4_ZEROS
    assert sgemv.sgemv_q4_desc_from_header(blob).as_dict() == d.as_dict()


def test_scale_types():
    torch = pytest.importorskip("torch")
    q, s, z = problem(3, 20, 200, 64)
    sb = torch.from_numpy(s.astype(np.float32)).bfloat16()
    raw = sb.view(torch.int16).numpy().view(np.uint16)
    d, blob = sgemv.sgemv_q4_pack(q, sb, z, 64)
    assert d.flags & sgemv.SGEMV_Q4_BF16_SCALES
    assert np.array_equal(blob, oracle.q4_pack_spec([(q, raw, z)], 64, bf16_scales=True))
    assert np.array_equal(sgemv.sgemv_q4_pack(q, raw, z, 64, bf16_scales=True)[1], blob)
    d2, blob2 = sgemv.sgemv_q4_pack(torch.from_numpy(q), torch.from_numpy(s), torch.from_numpy(z), 64)
    assert np.array_equal(blob2, sgemv.sgemv_q4_pack(q, s, z, 64)[1])
    assert not d2.flags & sgemv.SGEMV_Q4_BF16_SCALES


def test_layout_golden():
    """A few bytes by hand: the first word of output 0 holds inputs 0..7 as
    nibbles 0, 2, 4, 6, 1, 3, 5, 7 from the low end."""
    q = np.zeros((17, 130), dtype=np.uint8)
    q[0, :8] = [1, 2, 3, 4, 5, 6, 7, 8]
    q[0, 8] = 9          # lane 16 of the cell
    q[0, 32] = 10        # second word of lane 0
    q[16, 129] = 11      # second tile, second block, lane 0, element 1: nibble 4
    s = np.full((17, 2), 1.0, dtype=np.float16)
    d, b = sgemv.sgemv_q4_pack(q, s)
    word = lambda at: int(b[at:at + 4].view(np.uint32)[0])  # noqa: E731
    assert word(256) == 0x86427531
    assert word(256 + 16 * 16) == 9
    assert word(256 + 4) == 10
    assert word(256 + 3 * 1024) == 11 << 16
    assert b[d.s_off:d.s_off + 32].view(np.uint16).tolist() == [0x3C00] * 16


def test_oracle_product_exact_rationals():
    rng = np.random.default_rng(5)
    N, K, group = 3, 70, 32
    q, s, z = problem(6, N, K, group)
    x = rng.integers(-8, 9, (2, K)) / 4.0
    y = oracle.q4_product(x, q, s, z, group, bias=np.arange(N) / 8.0)
    for m in range(2):
        for n in range(N):
            want = Fraction(n, 8) + sum(Fraction(float(s[n, k // group])) * (int(q[n, k]) - int(z[n, k // group]))
                                        * Fraction(float(x[m, k])) for k in range(K))
            assert abs(y[m, n] - float(want)) < 1e-12
    one = np.zeros((1, K)); one[0, 33] = 1.0
    assert np.allclose(oracle.q4_product(one, q, s, None, group)[0], s[:, 1].astype(float) * (q[:, 33].astype(float) - 8))


def test_oracle_norm_closed_forms():
    v = np.array([[3.0, -4.0, 0.0, 0.0], [1.0, 1.0, 1.0, 1.0]])
    assert np.allclose(oracle.norm(v)[0], v[0] / 2.5)
    assert np.allclose(oracle.norm(v[:1] + 7.0, center=True), oracle.norm(v[:1] - v[:1].mean()))
    assert np.allclose(oracle.norm(v, weight=np.zeros(4), plus_one=True), oracle.norm(v))
    r, x = oracle.block_norm(v, y=v, gate=np.full(4, 2.0), scale=0.5)
    assert np.allclose(r, 2 * v) and np.allclose(x, oracle.norm(v))
    assert np.allclose(oracle.gate_function([0.0, 50.0, -50.0], "silu"), [0.0, 50.0, 0.0], atol=1e-18)
    assert np.allclose(oracle.gate_function([1.0], "gelu"), 0.8413447460685429)
    assert np.array_equal(oracle.gate_function([-1.0, 2.0], "relu"), [0.0, 2.0])


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_packer_refusals():
    q, s, z = problem(7, 16, 128, 64)
    L = sgemv.lib()

    def raw(q=q, s=s, z=z, N=16, K=128, group=64, flags=2, cap=None, gated=False):
        d = E.Q4Desc()
        out = np.zeros(8192, dtype=np.uint8)
        p = lambda a: None if a is None else a.ctypes.data  # noqa: E731
        cap = out.nbytes if cap is None else cap
        if gated:
            return L.sgemv_q4_pack_gated(p(q), p(s), p(z), p(q), p(s), p(z), N, K, group, flags, out.ctypes.data, cap, d)
        return L.sgemv_q4_pack(p(q), p(s), p(z), N, K, group, flags, out.ctypes.data, cap, d)

    assert raw() == E.SGEMV_OK and raw(gated=True) == E.SGEMV_OK
    assert raw(z=None, flags=0) == E.SGEMV_OK
    assert raw(q=None) == raw(s=None) == raw(z=None) == E.SGEMV_EINVAL
    for group in (0, -32, 16, 48, 256):
        assert raw(group=group) == E.SGEMV_EINVAL
    assert raw(flags=8) == raw(flags=3) == E.SGEMV_EINVAL      # unknown, and a lone matrix is not gated
    assert raw(N=0) == raw(K=0) == raw(N=E.SGEMV_MAX_N + 1) == raw(K=E.SGEMV_MAX_K + 1) == E.SGEMV_ESIZE
    assert raw(cap=255) == E.SGEMV_ESIZE
    for a, v in ((q, 16), (z, 16)):
        b = a.copy(); b[-1, -1] = v
        assert raw(**{"q" if a is q else "z": b}) == E.SGEMV_EINVAL
    for v in (np.inf, np.nan):
        b = s.copy(); b[3, 1] = v
        assert raw(s=b) == E.SGEMV_EINVAL
    b = s.copy().view(np.uint16); b[3, 1] = 0x7F80              # a bf16 infinity
    assert raw(s=b, flags=2 | 4) == E.SGEMV_EINVAL
    for args in ((q, s[:, :1], z), (q, s, z[:8]), (q.astype(np.int32), s, z), (q, s.astype(np.float32), z), (q[0], s, z)):
        with pytest.raises(ValueError):
            sgemv.sgemv_q4_pack(*args, 64)
    with pytest.raises(ValueError):
        sgemv.sgemv_q4_pack_gated((q, s, z), (q, s, None), 64)
    with pytest.raises(ValueError):
        sgemv.sgemv_q4_pack_gated((q, s, z), (q[:8], s[:8], z[:8]), 64)
    with pytest.raises(sgemv.SgemvError):
        sgemv.sgemv_q4_pack(q, s, z, 0)


def test_header_refusals():
    q, s, z = problem(8, 16, 128, 64)
    d, blob = sgemv.sgemv_q4_pack(q, s, z, 64)
    for off in (0, 4, 8, 12, 16, 24, 32, 40, 48, 56, 64, 72):
        b = blob.copy(); b[off] ^= 0x10
        with pytest.raises(sgemv.SgemvError):
            sgemv.sgemv_q4_desc_from_header(b)
    b = blob.copy(); b[20] |= 8
    with pytest.raises(sgemv.SgemvError):
        sgemv.sgemv_q4_desc_from_header(b)
    with pytest.raises(sgemv.SgemvError):
        sgemv.sgemv_q4_desc_from_header(blob[:79])
    with pytest.raises(sgemv.SgemvError):   # a blob of the sparse calls
        sgemv.sgemv_q4_desc_from_header(oracle.pack_spec(*_sparse(), 512))


def _sparse():
    import synth
    return synth.random_int4_problem(1, 512, 128)


def test_run_refusals():
    L = sgemv.lib()
    q, s, z = problem(9, 40, 200, 32)
    d, _ = sgemv.sgemv_q4_pack(q, s, z, 32)
    dg, _ = sgemv.sgemv_q4_pack_gated((q, s, z), (q, s, z), 32)

    def run(d=d, packed=FAKE, x=FAKE, xt=0, M=1, ldx=200, bias=None, y=FAKE, yt=0, ldy=40):
        return L.sgemv_q4_run(d, packed, x, xt, M, ldx, bias, y, yt, ldy, None)

    assert run(d=None) == run(packed=None) == run(x=None) == run(y=None) == E.SGEMV_EINVAL
    assert run(d=dg) == run(xt=2) == run(xt=3) == run(xt=-1) == run(yt=1) == run(yt=3) == run(xt=1, yt=0) == E.SGEMV_EINVAL
    assert run(M=0) == run(M=17) == run(M=-1) == run(ldx=199) == run(ldy=39) == E.SGEMV_ESIZE
    assert run(packed=FAKE + 128) == run(x=FAKE + 1) == run(y=FAKE + 1) == run(y=FAKE + 2, yt=2) == E.SGEMV_EALIGN
    assert run(bias=FAKE + 1) == E.SGEMV_EALIGN
    # y inside x's rows, x inside y's, y over the blob or the bias, columns that meet
    assert run(packed=FAKE << 2, y=FAKE + 398) == run(packed=FAKE << 2, x=FAKE + 78) == E.SGEMV_EINVAL
    assert run(y=FAKE + int(d.total_bytes) - 2, x=FAKE << 2) == run(packed=FAKE << 2, x=FAKE << 3, bias=FAKE) == E.SGEMV_EINVAL
    assert run(packed=FAKE << 2, M=4, ldx=512, ldy=512, y=FAKE + 398) == E.SGEMV_EINVAL
    assert run(packed=FAKE << 2, M=4, ldx=512, ldy=512, y=FAKE + 1024 - 78) == E.SGEMV_EINVAL
    bad = E.Q4Desc(**d.as_dict()); bad.s_off += 256
    assert run(d=bad) == E.SGEMV_EINVAL
    bad = E.Q4Desc(**d.as_dict()); bad.K = 0
    assert run(d=bad) == E.SGEMV_ESIZE

    def gated(d=dg, act=0, M=1, xt=0, yt=0, bg=None, bu=None):
        return L.sgemv_q4_run_gated(d, FAKE, FAKE, xt, M, 200, bg, bu, act, FAKE, yt, 40, None)

    assert gated(d=d) == gated(act=3) == gated(act=-1) == gated(xt=2) == gated(yt=1) == E.SGEMV_EINVAL
    assert gated(M=17) == E.SGEMV_ESIZE
    assert gated(bu=FAKE + 1) == E.SGEMV_EALIGN


def test_device_packer_refusals():
    L = sgemv.lib()

    def pack(q=FAKE, s=FAKE, z=FAKE, qu=None, su=None, zu=None, N=16, K=128, group=64, flags=2, out=FAKE, cap=1 << 20):
        return L.sgemv_q4_pack_device(q, s, z, qu, su, zu, N, K, group, flags, out, cap, None, None)

    assert pack(q=None) == pack(s=None) == pack(z=None) == pack(out=None) == E.SGEMV_EINVAL
    assert pack(group=48) == pack(flags=16) == pack(flags=3) == pack(flags=3, qu=FAKE, su=FAKE) == E.SGEMV_EINVAL
    assert pack(N=0) == pack(K=1 << 17) == pack(cap=1791) == E.SGEMV_ESIZE   # 1792 needed
    assert pack(out=FAKE + 16) == pack(s=FAKE + 1) == E.SGEMV_EALIGN
    torch = pytest.importorskip("torch")
    q, s, z = (torch.from_numpy(a) for a in problem(1, 16, 128, 64))
    for match, f in (("GPU tensor", lambda: sgemv.sgemv_q4_pack_device(q, s, z, group=64)),
                     ("codes", lambda: sgemv.sgemv_q4_pack_device(q.int(), s, z, group=64)),
                     ("scales", lambda: sgemv.sgemv_q4_pack_device(q, s.float(), z, group=64)),
                     ("both", lambda: sgemv.sgemv_q4_pack_device(q, s, z, up=(q, s, None), group=64))):
        with pytest.raises(ValueError, match=match):
            f()


def norm_args(**kw):
    f = dict(rows=4, D=64, flags=0, residual=FAKE, y=0, gate=0, post_weight=0, post_bias=0, weight=0, bias=0,
             residual_out=0, x=FAKE + (1 << 16), ld_residual=64, ld_y=64, ld_gate=0, ld_residual_out=64, ld_x=64,
             scale=1.0, eps=1e-6, residual_type=0, y_type=0, w_type=0, x_type=0)
    assert set(kw) <= set(f)
    f.update(kw)
    return sgemv._NORM.pack(*f.values())


def norm_call(**kw):
    return sgemv.lib().sgemv_block_norm(norm_args(**kw), None)


def test_norm_refusals():
    assert sgemv.lib().sgemv_block_norm(None, None) == E.SGEMV_EINVAL
    Y = FAKE + (2 << 16)
    for kw in (dict(residual=0), dict(x=0), dict(flags=8), dict(flags=1), dict(gate=Y), dict(y=Y, post_weight=FAKE),
               dict(y=Y, post_bias=FAKE), dict(residual_type=3), dict(y_type=-1), dict(w_type=3), dict(x_type=7),
               dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert norm_call(**kw) == E.SGEMV_EINVAL, kw
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(D=0), dict(D=65537, ld_residual=1 << 17, ld_x=1 << 17),
               dict(ld_residual=63), dict(ld_x=63), dict(y=Y, ld_y=63), dict(y=Y, gate=Y, ld_gate=1),
               dict(residual_out=Y, ld_residual_out=0), dict(ld_x=1 << 40)):
        assert norm_call(**kw) == E.SGEMV_ESIZE, kw
    for kw in (dict(residual=FAKE + 1), dict(x=FAKE + 5), dict(x=FAKE + (1 << 16) + 2, x_type=2),
               dict(y=Y + 1), dict(weight=Y + 2, w_type=2), dict(residual_out=Y + 1)):
        assert norm_call(**kw) == E.SGEMV_EALIGN, kw


def test_norm_overlaps_are_refused():
    R, X = FAKE, FAKE + (1 << 16)
    for kw in (dict(x=R + 2), dict(x=R - 2), dict(x=R + 64 * 2 * 3 + 126),        # shifted views of residual
               dict(x=R, x_type=2),                                               # another element size
               dict(x=R, ld_x=128),                                               # another stride
               dict(residual_out=X), dict(residual_out=X + 64), dict(residual_out=R, x=R),
               dict(weight=X), dict(bias=X + 2), dict(y=R + 4096, gate=X, ld_gate=0),
               dict(y=X + 64, ld_y=64),
               dict(x=R + 126, ld_x=128, ld_residual=128),                        # columns that meet
               dict(x=R + 132, ld_x=128, ld_residual=128)):                       # ... and wrap into the next row
        assert norm_call(**kw) == E.SGEMV_EINVAL, kw


def test_norm_of_no_rows():
    assert norm_call(rows=0) == E.SGEMV_OK


# ---------------------------------------------------------------------------
# the binding's own checks
# ---------------------------------------------------------------------------
def test_binding_refuses_host_tensors_and_wrong_operands():
    torch = pytest.importorskip("torch")
    q, s, z = problem(10, 40, 200, 64)
    m = sgemv.Q4Matrix(q, s, z, group=64, device="cpu")
    x, y = torch.zeros(3, 200, dtype=torch.float16), torch.zeros(3, 40, dtype=torch.float16)
    run = lambda x=x, y=y, **kw: sgemv.sgemv_q4_run(m.desc, m.blob, x, y, **kw)  # noqa: E731
    for match, f in (("GPU tensor", lambda: run()), ("dtype", lambda: run(x=x.float())), ("dtype", lambda: run(y=y.bfloat16())),
                     ("dtype", lambda: run(x=x.double())), ("shape", lambda: run(x=x[:, :199])),
                     ("shape", lambda: run(y=y[:2])), ("contiguous", lambda: run(x=torch.zeros(200, 3).half().t())),
                     ("rows overlap", lambda: run(x=torch.zeros(1, 200).half().expand(3, 200))),
                     ("dtype", lambda: run(bias=torch.zeros(40))), ("shape", lambda: run(bias=torch.zeros(39).half())),
                     ("packed", lambda: sgemv.sgemv_q4_run(m.desc, m.blob[:-1], x, y)),
                     ("act", lambda: sgemv.sgemv_q4_run_gated(m.desc, m.blob, x, y, act="tanh")),
                     ("one row", lambda: run(y=y[0])), ("torch tensor", lambda: run(x=np.zeros((3, 200))))):
        with pytest.raises(ValueError, match=match):
            f()


def test_norm_binding_checks():
    torch = pytest.importorskip("torch")
    r, x = torch.zeros(3, 50), torch.zeros(3, 50).half()
    f = lambda *a, **kw: sgemv.sgemv_block_norm(*a, **kw)  # noqa: E731
    for match, g in (("GPU tensor", lambda: f(x, r)), ("needs y", lambda: f(x, r, gate=r)),
                     ("needs y", lambda: f(x, r, post_norm=True)), ("post_weight", lambda: f(x, r, r, post_weight=r[0], post_norm=False)),
                     ("residual_out", lambda: f(x, r, r, x)), ("shape", lambda: f(x[:2], r)), ("shape", lambda: f(x, r, r[:, :49])),
                     ("dtype", lambda: f(x, r.double())), ("differs", lambda: f(x, r, weight=r[0], bias=x[0])),
                     ("shape", lambda: f(x, r, weight=r[0, :49])), ("gate", lambda: f(x, r, r, gate=x))):
        with pytest.raises(ValueError, match=match):
            g()


def test_binding_refuses_sizes_beyond_int32():
    """The C calls take rows, row strides and sizes as int32: larger ones are
    refused, not cut off (2^32 + 16 would arrive as 16)."""
    torch = pytest.importorskip("torch")
    q, s, z = problem(11, 16, 32, 32)
    desc, blob = sgemv.sgemv_q4_pack(q, s, z, 32)
    packed = torch.from_numpy(blob)
    big = 1 << 32

    def meta(rows, n, ld, dtype=torch.float16):
        return torch.empty_strided((rows, n), (ld, 1), dtype=dtype, device="meta")
    x, y = meta(2, 32, 32), meta(2, 16, 16)
    for f in (lambda: sgemv.sgemv_q4_run(desc, packed, meta(2, 32, big + 32), y),
              lambda: sgemv.sgemv_q4_run(desc, packed, x, meta(2, 16, big + 16)),
              lambda: sgemv.sgemv_q4_run(desc, packed, x, meta(2, 16, 1 << 31)),
              lambda: sgemv.sgemv_q4_run(desc, packed, meta(big + 1, 32, 32), meta(big + 1, 16, 16)),
              lambda: sgemv.sgemv_q4_pack(q, s, z, big + 32),
              lambda: sgemv.sgemv_q4_pack_device(meta(big + 16, 32, 32, torch.uint8), meta(big + 16, 1, 1)),
              lambda: sgemv.sgemv_block_norm(meta(1, big + 8, big + 8), meta(1, big + 8, big + 8))):
        with pytest.raises(sgemv.SgemvError) as e:
            f()
        assert e.value.status == sgemv.SGEMV_ESIZE


def test_norm_binding_refuses_a_gate_without_dimensions():
    torch = pytest.importorskip("torch")
    r = torch.zeros(3, 50)
    with pytest.raises(ValueError, match="gate"):
        sgemv.sgemv_block_norm(r, r, r, gate=torch.tensor(1.0))
    none = torch.zeros(0, 50)
    with pytest.raises(ValueError, match="GPU tensor"):
        sgemv.sgemv_block_norm(none, none, none, gate=torch.zeros(60).expand(0, 60))


def test_packers_refuse_a_scale_type_that_the_scales_contradict():
    """bf16_scales says what uint16 scales hold; scales that carry a type of
    their own are never read as another, in either projection of a pair."""
    torch = pytest.importorskip("torch")
    q, s, z = problem(12, 17, 130, 64)
    h, b = torch.from_numpy(s), torch.from_numpy(s.astype(np.float32)).bfloat16()
    raw = bits(s)
    for scales, said in ((s, True), (h, True), (b, False)):
        with pytest.raises(ValueError, match="scales"):
            sgemv.sgemv_q4_pack(q, scales, z, 64, bf16_scales=said)
        with pytest.raises(ValueError, match="scales"):
            sgemv.Q4Matrix(q, scales, z, group=64, device="cpu", bf16_scales=said)
        for pair in (((q, scales, z), (q, raw, z)), ((q, raw, z), (q, scales, z))):
            with pytest.raises(ValueError, match="scales"):
                sgemv.sgemv_q4_pack_gated(*pair, 64, bf16_scales=said)
    for said in (None, False, True):
        with pytest.raises(ValueError, match="scales"):
            sgemv.sgemv_q4_pack_gated((q, b, z), (q, h, z), 64, bf16_scales=said)
    # what agrees is taken: a type said twice, bits beside a typed projection when it is said what they hold
    for scales, said in ((s, False), (h, False), (b, True)):
        want = sgemv.sgemv_q4_pack(q, scales, z, 64)
        got = sgemv.sgemv_q4_pack(q, scales, z, 64, bf16_scales=said)
        assert got[0].as_dict() == want[0].as_dict() and np.array_equal(got[1], want[1])
    got = sgemv.sgemv_q4_pack_gated((q, s, z), (q, raw, z), 64, bf16_scales=False)
    assert np.array_equal(got[1], sgemv.sgemv_q4_pack_gated((q, s, z), (q, s, z), 64)[1])


@pytest.mark.parametrize("when", ["before", "after"])
def test_first_calls_from_two_threads(monkeypatch, when):
    """The binding's tables are filled on the first call.  Calls that come
    from another thread while that happens are answered like any other: here
    they are made just before and just after the type table is filled."""
    torch = pytest.importorskip("torch")
    import threading
    q, s, z = problem(13, 16, 32, 32)
    desc, blob = sgemv.sgemv_q4_pack(q, s, z, 32)
    packed, x, y = torch.from_numpy(blob), torch.zeros(2, 32).half(), torch.zeros(2, 16).half()
    started, other = [], []

    def second():
        for call in (lambda: sgemv.sgemv_q4_run(desc, packed, x, y), lambda: sgemv.sgemv_block_norm(x, x)):
            try:
                call()
            except Exception as e:   # noqa: BLE001
                other.append(e)

    def from_another_thread():
        if not started:
            started.append(True)
            t = threading.Thread(target=second)
            t.start()
            t.join()

    class Table(dict):
        def update(self, *a, **kw):
            if when == "before":
                from_another_thread()
            super().update(*a, **kw)
            if when == "after":
                from_another_thread()

    monkeypatch.setattr(sgemv, "_TYPES", Table())
    for name in ("_torch", "_raw_stream", "_device_now"):
        monkeypatch.setattr(sgemv, name, None)
    sgemv._load_torch()
    assert len(other) == 2
    for e in other:   # host tensors: both calls are valid up to that check
        assert type(e) is ValueError and "GPU tensor" in str(e), repr(e)
    assert sgemv._raw_stream is not None and sgemv._device_now is not None


def test_gated_refusals_name_the_gated_call_and_its_output():
    torch = pytest.importorskip("torch")
    part = problem(14, 16, 32, 32)
    desc, blob = sgemv.sgemv_q4_pack_gated(part, part, 32)
    packed = torch.from_numpy(blob)
    far = torch.empty_strided((2, 32), ((1 << 32) + 32, 1), dtype=torch.float16, device="meta")
    with pytest.raises(sgemv.SgemvError, match="sgemv_q4_run_gated: ldx"):
        sgemv.sgemv_q4_run_gated(desc, packed, far, torch.zeros(2, 16).half())
    x = torch.zeros(2, 32).half()
    for h in (torch.zeros(2, 15).half(), torch.zeros(3, 16).half(), torch.zeros(2, 16).double(), torch.zeros(2, 16).bfloat16(),
              torch.zeros(16, 2).half().t()):
        with pytest.raises(ValueError, match="^h: "):
            sgemv.sgemv_q4_run_gated(desc, packed, x, h)
        with pytest.raises(ValueError, match="^y: "):
            sgemv.sgemv_q4_run(desc, packed, x, h)


def test_device_packer_refuses_inputs_inside_the_blob():
    """The blob is written while the inputs are read: an input that shares
    bytes with it is refused."""
    L = sgemv.lib()
    d, total = E.Q4Desc(), {}
    for flags in (2, 3):
        fn, n = (L.sgemv_q4_pack_gated, 6) if flags & 1 else (L.sgemv_q4_pack, 3)
        assert fn(*[None] * n, 16, 128, 64, flags, None, 0, d) == E.SGEMV_OK
        total[flags] = int(d.total_bytes)
    out, far = FAKE, [FAKE << k for k in range(1, 7)]
    size = {"q": 16 * 128, "s": 16 * 2 * 2, "z": 16 * 2}

    def pack(flags, **at):
        p = [at.get(k, far[i]) for i, k in enumerate(("q", "s", "z", "qu", "su", "zu"))]
        if not flags & 1:
            p[3:] = [None] * 3
        return L.sgemv_q4_pack_device(*p, 16, 128, 64, flags, out, 1 << 20, None, None)

    for flags, names in ((2, "q s z"), (3, "q s z qu su zu")):
        for name in names.split():
            for at in (out, out + 64, out + total[flags] - 2, out - size[name[0]] + 2):
                assert pack(flags, **{name: at}) == E.SGEMV_EINVAL, (flags, name, at - out)


def test_oracle_gelu_far_out():
    """v Phi(v) with Phi from tables: relative accuracy where 1 + erf cancels."""
    for v, phi in ((-3.0, 1.3498980316300945e-03), (-6.0, 9.865876450376981e-10), (-10.0, 7.619853024160527e-24)):
        assert abs(float(oracle.gate_function([v], "gelu")[0]) / (v * phi) - 1) < 1e-12


def test_binding_refuses_operands_without_dimensions_and_other_kinds():
    torch = pytest.importorskip("torch")
    q, s, z = problem(15, 16, 32, 32)
    desc, blob = sgemv.sgemv_q4_pack(q, s, z, 32)
    packed, x, y = torch.from_numpy(blob), torch.zeros(2, 32).half(), torch.zeros(2, 16).half()
    point, r = torch.tensor(1.0).half(), torch.zeros(3, 50)
    qt, st, zt = torch.from_numpy(q), torch.from_numpy(s), torch.from_numpy(z)
    for match, f in (("^x: ", lambda: sgemv.sgemv_q4_run(desc, packed, point, y)),
                     ("^y: ", lambda: sgemv.sgemv_q4_run(desc, packed, x, point)),
                     ("^x: ", lambda: sgemv.sgemv_q4_run(desc, packed, None, y)),
                     ("^bias: ", lambda: sgemv.sgemv_q4_run(desc, packed, x, y, bias=point)),
                     ("^packed: ", lambda: sgemv.sgemv_q4_run(desc, blob, x, y)),
                     ("^residual: ", lambda: sgemv.sgemv_block_norm(r, torch.tensor(1.0))),
                     ("^x: ", lambda: sgemv.sgemv_block_norm(torch.tensor(1.0), r)),
                     ("^y: ", lambda: sgemv.sgemv_block_norm(r, r, torch.tensor(1.0))),
                     ("^weight: ", lambda: sgemv.sgemv_block_norm(r, r, weight=torch.tensor(1.0))),
                     ("^residual_out: ", lambda: sgemv.sgemv_block_norm(r, r, r, torch.tensor(1.0))),
                     ("^weight codes: ", lambda: sgemv.sgemv_q4_pack_device(q, st, zt, group=32)),
                     ("^weight codes: ", lambda: sgemv.sgemv_q4_pack_device(qt[0], st, zt, group=32)),
                     ("^weight zeros: ", lambda: sgemv.sgemv_q4_pack_device(qt, st, z, group=32)),
                     ("^up codes: ", lambda: sgemv.sgemv_q4_pack_device(qt, st, zt, up=(q, st, zt), group=32)),
                     ("^up scales: ", lambda: sgemv.sgemv_q4_pack_device(qt, st, zt, up=(qt, s, zt), group=32))):
        with pytest.raises(ValueError, match=match):
            f()
