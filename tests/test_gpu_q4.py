"""The 4-bit products that read every weight and the gated pair against
their float64 definitions.

Tolerance.  A product's sum has at most 128 terms a group on the matrix
cores, then one term a group and one a wavefront (at most 16), in fp32; with
each addition off by at most 2^-23 of the running magnitude (rounding or
truncation), |y - y_ref| <= (128 + groups + 16) 2^-23 E, with E = sum |s|
|q - z| |x| for fp16 activations and sum |s| (q + z + 32) |x| for bf16 ones
(codes and zero-points go in with 16 added).  The bias adds one fp32 rounding
and the output type half a step (eps / 2), for fp16 at least half its
smallest subnormal."""
import numpy as np
import pytest

import oracle
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def problem(seed, N, K, group, zeros=True, bf16_scales=False):
    rng = np.random.default_rng(seed)
    g = -(-K // group)
    q = rng.integers(0, 16, (N, K), dtype=np.uint8)
    s = torch.from_numpy(rng.uniform(0.003, 0.02, (N, g)).astype(np.float32)).to(T["bf16" if bf16_scales else "f16"])
    z = rng.integers(0, 16, (N, g), dtype=np.uint8) if zeros else None
    return q, s, z


def f64(t):
    return t.detach().double().cpu().numpy()


def activations(seed, M, K, t):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.01, 20.0, 1.0)
    return torch.from_numpy(x.astype(np.float32)).to(T[t])


def accumulation(x, part, group):
    """Bound on the fp32 error of a product, without bias and output."""
    q, s, z = part
    bf = x.dtype == torch.bfloat16
    depth = 128 + -(-q.shape[1] // group) + 16
    return depth * 2.0 ** -23 * oracle.q4_scale(f64(x), q, f64(s), z, group, 16.0 if bf else 0.0)


def rounding(y, t):
    return np.abs(y) * torch.finfo(T[t]).eps / 2 + (2.0 ** -25 if t == "f16" else 2.0 ** -134)


def check(got, ref, tol, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    over = np.abs(got - ref) - tol
    assert not (over > 0).any(), f"{what}: {int((over > 0).sum())} of {got.size} outside, worst by {over.max():.3e}"


def run_product(x, part, group, yt, bias=None, ldy=None):
    from activation_sparse_bit_amd import sgemv
    m = sgemv.Q4Matrix(*part, group=group, device="cuda:0")
    M, N = x.shape[0], m.N
    y = torch.full((M + 1, ldy or N), float("nan"), dtype=T[yt], device="cuda:0")
    b = None if bias is None else bias.cuda()
    sgemv.sgemv_q4_run(m.desc, m.blob, x.cuda(), y[:M, :], bias=b)
    torch.cuda.synchronize()
    assert torch.isnan(y[M:]).all() and torch.isnan(y[:, N:]).all()   # nothing beyond the output
    return y[:M, :N]


def check_product(seed, N, K, M, group, xt, yt, zeros, bf16_scales, bias, ldy=None):
    part = problem(seed, N, K, group, zeros, bf16_scales)
    x = activations(seed + 1, M, K, xt)
    b = torch.from_numpy(np.random.default_rng(seed + 2).standard_normal(N).astype(np.float32)).to(T[xt]) if bias else None
    got = run_product(x, part, group, yt, b, ldy)
    ref = oracle.q4_product(f64(x), part[0], f64(part[1]), part[2], group, None if b is None else f64(b))
    tol = accumulation(x, part, group) + rounding(ref, yt) + (np.abs(ref) * 2.0 ** -23 if bias else 0)
    check(got, ref, tol * (1 + 2.0 ** -7), f"N={N} K={K} M={M}")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
@pytest.mark.parametrize("N,K,M", [(1, 1, 1), (15, 31, 1), (16, 32, 2), (17, 33, 3), (64, 127, 4), (65, 128, 5),
                                   (33, 129, 8), (48, 500, 9), (130, 1111, 16), (257, 2048, 1), (96, 4000, 12),
                                   (40, 8200, 7)])
def test_product_sizes(N, K, M, xt, group):
    seed = N * 7919 + K * 31 + M
    check_product(seed, N, K, M, group, xt, "f32" if (N + K) % 2 else xt, zeros=seed % 3 != 0,
                  bf16_scales=seed % 2 == 0, bias=seed % 5 < 2)


@pytest.mark.parametrize("M", range(1, 17))
@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_product_rows(M, xt):
    check_product(100 + M, 80, 640, M, 64, xt, "f32", True, False, True)


@pytest.mark.parametrize("N,K,M,group,xt", [(2048, 2048, 1, 128, "f16"), (4096, 14336, 1, 128, "f16"),
                                            (1024, 4096, 16, 32, "bf16"), (20001, 1024, 4, 64, "f16"),
                                            (70, 65536, 3, 128, "bf16")])
def test_product_larger(N, K, M, group, xt):
    check_product(3, N, K, M, group, xt, xt, True, False, False)


@pytest.mark.parametrize("xt", ["f16", "bf16"])
@pytest.mark.parametrize("N,K,M,group", [(8300, 384, 3, 64), (8300, 384, 6, 32), (8300, 384, 16, 128), (16500, 300, 16, 32),
                                         (16500, 1024, 9, 64), (33000, 640, 2, 32), (33000, 1000, 12, 128),
                                         (5000, 4224, 16, 64), (300, 4224, 16, 32), (300, 8192, 8, 128)])
def test_product_tiles_and_wavefronts(N, K, M, group, xt):
    """Every number of tiles a workgroup has (1, 2, 4) and of wavefronts."""
    check_product(N + K, N, K, M, group, xt, "f32", True, False, True)


@pytest.mark.parametrize("M,xt", [(2, "f16"), (7, "bf16"), (16, "bf16"), (16, "f16")])
@pytest.mark.parametrize("N,group", [(8200, 128), (20000, 32)])
def test_product_streamed(N, M, xt, group):
    """Matrices large enough for their codes to be read past the caches."""
    K = -(-(96 << 21) // N // 128) * 128 + 37
    gen = torch.Generator(device="cuda:0").manual_seed(N)
    from activation_sparse_bit_amd import sgemv
    g = -(-K // group)
    q = torch.randint(0, 16, (N, K), dtype=torch.uint8, device="cuda:0", generator=gen)
    s = (0.01 + 0.01 * torch.rand(N, g, device="cuda:0", generator=gen)).half()
    z = torch.randint(0, 16, (N, g), dtype=torch.uint8, device="cuda:0", generator=gen)
    m = sgemv.Q4Matrix(q, s, z, group=group)
    assert m.desc.w_bytes >= 96 << 20
    x = activations(5, M, K, xt)
    y = torch.empty(M, N, dtype=torch.float32, device="cuda:0")
    sgemv.sgemv_q4_run(m.desc, m.blob, x.cuda(), y)
    rows = np.array(sorted({0, 1, 15, 16, 33, 63, 64, N // 2, N - 17, N - 2, N - 1}))
    part = (q[rows].cpu().numpy(), s[rows].cpu(), z[rows].cpu().numpy())
    ref = oracle.q4_product(f64(x), part[0], f64(part[1]), part[2], group)
    check(y[:, rows], ref, accumulation(x, part, group) + rounding(ref, "f32") * 1.01, f"N={N} K={K}")


@pytest.mark.parametrize("N,K,group", [(1, 1, 32), (16, 128, 128), (17, 129, 32), (100, 1000, 64), (333, 257, 128)])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("bf16", [False, True])
def test_device_packer_makes_the_host_blob(N, K, group, zeros, bf16):
    from activation_sparse_bit_amd import sgemv
    a, b = problem(1, N, K, group, zeros, bf16), problem(2, N, K, group, zeros, bf16)
    dev = lambda p: tuple(None if t is None else torch.as_tensor(t).cuda() for t in p)  # noqa: E731
    for host, gpu in ((sgemv.sgemv_q4_pack(*a, group), sgemv.sgemv_q4_pack_device(*dev(a), group=group)),
                      (sgemv.sgemv_q4_pack_gated(a, b, group), sgemv.sgemv_q4_pack_device(*dev(a), up=dev(b), group=group))):
        assert host[0].as_dict() == gpu[0].as_dict()
        assert np.array_equal(host[1], gpu[1].cpu().numpy())
    q, s, z = dev(a)
    q = q.clone(); q[-1, -1] = 16
    with pytest.raises(sgemv.SgemvError):
        sgemv.sgemv_q4_pack_device(q, s, z, group=group)
    s = s.clone(); s[0, 0] = float("inf")
    with pytest.raises(sgemv.SgemvError):
        sgemv.sgemv_q4_pack_device(dev(a)[0], s, z, group=group)


@pytest.mark.parametrize("xt", ["f16", "bf16"])
@pytest.mark.parametrize("off,pad", [(0, 5), (1, 0), (3, 7)])
def test_strides_and_alignment(xt, off, pad):
    """Rows of a wider buffer at any element: x, bias and y start off a
    16-byte boundary; what lies between the rows of y stays."""
    from activation_sparse_bit_amd import sgemv
    N, K, M, group = 50, 300, 6, 64
    part = problem(11, N, K, group)
    x = activations(12, M, K, xt)
    m = sgemv.Q4Matrix(*part, group=group, device="cuda:0")
    wide = torch.full((M * (K + pad) + off + 8,), float("nan"), dtype=T[xt], device="cuda:0")
    xv = wide[off:off + M * (K + pad)].view(M, K + pad)[:, :K]
    xv.copy_(x)
    out = torch.full((M, N + pad + 9), 7.0, dtype=T[xt], device="cuda:0")
    bias = torch.zeros(N + 3, dtype=T[xt], device="cuda:0")[off:off + N]
    sgemv.sgemv_q4_run(m.desc, m.blob, xv, out[:, 1:1 + N], bias=bias)
    ref = oracle.q4_product(f64(x), part[0], f64(part[1]), part[2], group)
    check(out[:, 1:1 + N], ref, accumulation(x, part, group) + rounding(ref, xt) * (1 + 2.0 ** -7))
    assert (out[:, :1] == 7).all() and (out[:, 1 + N:] == 7).all()


def test_operands_in_one_buffer():
    """x and y as columns of one wider buffer."""
    from activation_sparse_bit_amd import sgemv
    part = problem(15, 70, 200, 64)
    x = activations(16, 5, 200, "f16")
    m = sgemv.Q4Matrix(*part, group=64, device="cuda:0")
    wide = torch.full((5, 300), 3.0, dtype=torch.float16, device="cuda:0")
    wide[:, 75:275] = x.cuda()
    sgemv.sgemv_q4_run(m.desc, m.blob, wide[:, 75:275], wide[:, 3:73])
    ref = oracle.q4_product(f64(x), part[0], f64(part[1]), part[2], 64)
    check(wide[:, 3:73], ref, accumulation(x, part, 64) + rounding(ref, "f16") * 1.01)
    assert torch.equal(wide[:, 75:275].cpu(), x) and (wide[:, :3] == 3).all() and (wide[:, 275:] == 3).all()


def test_codes_equal_to_zero_points_give_zero():
    """q = z everywhere: exactly 0 for fp16 activations; for bf16 the sums of
    (16 + z) x and their correction cancel to accumulation error."""
    q, s, z = problem(21, 64, 700, 64)
    q = np.repeat(z, 64, axis=1)[:, :700].copy()
    x = activations(22, 3, 700, "f16")
    assert (run_product(x, (q, s, z), 64, "f32") == 0).all()
    xb = activations(22, 3, 700, "bf16")
    check(run_product(xb, (q, s, z), 64, "f32"), np.zeros((3, 64)), accumulation(xb, (q, s, z), 64))


@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_non_finite_rows_stay_apart(xt):
    """An infinity or a NaN in one row of x leaves the other rows as they
    are; in fp16 an infinity gives the infinity or NaN that the formula has."""
    part = problem(31, 48, 260, 64)
    x = activations(32, 6, 260, xt)
    clean = run_product(x, part, 64, "f32")
    x[1, 7], x[3, 259], x[4, 100] = float("inf"), float("nan"), float("-inf")
    got = run_product(x, part, 64, "f32")
    for m in (0, 2, 5):
        assert torch.equal(got[m], clean[m])
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[[1, 4]]).any()
    if xt == "f16":
        ref = oracle.q4_product(f64(x), part[0], f64(part[1]), part[2], 64)
        for m in (1, 4):
            assert np.array_equal(np.isnan(ref[m]), f64(torch.isnan(got[m])) > 0)
            fine = ~np.isnan(ref[m])
            assert np.array_equal(ref[m][fine], f64(got[m])[fine])


def test_small_and_large_activations():
    """fp16 subnormals and the largest fp16 values, bf16 far outside fp16's
    range."""
    part = problem(41, 32, 384, 128)
    rng = np.random.default_rng(42)
    for xt, mags in (("f16", (2.0 ** -24, 2.0 ** -16, 60000.0)), ("bf16", (1e-30, 1e-12, 1e20))):
        for mag in mags:
            x = torch.from_numpy((rng.uniform(-1, 1, (2, 384)) * mag).astype(np.float32)).to(T[xt])
            ref = oracle.q4_product(f64(x), part[0], f64(part[1]), part[2], 128)
            check(run_product(x, part, 128, "f32"), ref, accumulation(x, part, 128) + rounding(ref, "f32") * 1.01, str(mag))


def test_one_dimensional_row():
    from activation_sparse_bit_amd import sgemv
    part = problem(51, 100, 256, 128)
    x = activations(52, 1, 256, "f16")
    m = sgemv.Q4Matrix(*part, device="cuda:0")
    y = torch.empty(100, dtype=torch.float16, device="cuda:0")
    sgemv.sgemv_q4_run(m.desc, m.blob, x[0].cuda(), y)
    assert torch.equal(y, run_product(x, part, 128, "f16")[0])


# ---------------------------------------------------------------------------
# the gated pair
# ---------------------------------------------------------------------------
def check_gated(seed, N, K, M, group, xt, ht, act, zeros=True, bias=False):
    from activation_sparse_bit_amd import sgemv
    gate, up = problem(seed, N, K, group, zeros), problem(seed + 1, N, K, group, zeros)
    x = activations(seed + 2, M, K, xt) * 0.3
    rng = np.random.default_rng(seed + 3)
    bg, bu = [torch.from_numpy(rng.standard_normal(N).astype(np.float32)).to(T[xt]) for _ in range(2)] if bias else (None, None)
    m = sgemv.Q4Matrix.gated(gate, up, group=group, device="cuda:0")
    h = torch.full((M + 1, N), float("nan"), dtype=T[ht], device="cuda:0")
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    sgemv.sgemv_q4_run_gated(m.desc, m.blob, x.cuda(), h[:M], act=act, bias_gate=dev(bg), bias_up=dev(bu))
    torch.cuda.synchronize()
    assert torch.isnan(h[M]).all()
    n = lambda t: None if t is None else f64(t)  # noqa: E731
    g = oracle.q4_product(f64(x), gate[0], f64(gate[1]), gate[2], group, n(bg))
    u = oracle.q4_product(f64(x), up[0], f64(up[1]), up[2], group, n(bu))
    ref = oracle.gate_function(g, act) * u
    eg = accumulation(x, gate, group) + np.abs(g) * 2.0 ** -23
    eu = accumulation(x, up, group) + np.abs(u) * 2.0 ** -23
    # |act'| <= 1.13; exp and erf within 4 steps of 2^-24 of values near 1,
    # and the products and the quotient one each: 16 steps of |g| in all
    ea = 1.13 * eg + 16 * 2.0 ** -24 * np.abs(g)
    tol = ea * (np.abs(u) + eu) + np.abs(oracle.gate_function(g, act)) * eu + 2.0 ** -23 * np.abs(ref)
    check(h[:M], ref, tol * (1 + 2.0 ** -7) + rounding(ref, ht) * (1 + 2.0 ** -7), f"{act} N={N} K={K} M={M}")


@pytest.mark.parametrize("N,K,M,group,xt", [(8300, 384, 16, 64, "bf16"), (8300, 200, 11, 32, "f16"), (4200, 640, 2, 128, "f16")])
def test_gated_tiles(N, K, M, group, xt):
    check_gated(N, N, K, M, group, xt, "f32", "silu")


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("N,K,M,group,xt,ht", [(1, 1, 1, 128, "f16", "f32"), (16, 128, 4, 32, "bf16", "bf16"),
                                               (17, 300, 5, 64, "f16", "f16"), (100, 1000, 16, 32, "f16", "f32"),
                                               (333, 515, 9, 128, "bf16", "f32"), (1000, 4096, 1, 128, "f16", "f16")])
def test_gated_sizes(N, K, M, group, xt, ht, act):
    check_gated(N + K, N, K, M, group, xt, ht, act, zeros=N % 2 == 0, bias=K % 3 == 0)


def test_gated_saturates():
    """Gates far out on both sides: silu and gelu go to v and to 0."""
    from activation_sparse_bit_amd import sgemv
    N, K = 32, 128
    q = np.full((N, K), 8, dtype=np.uint8)
    q[:16, 0], q[16:, 0] = 15, 1
    one = np.full((N, 1), 1.0, dtype=np.float16)
    up = np.full((N, K), 8, dtype=np.uint8); up[:, 0] = 9
    m = sgemv.Q4Matrix.gated((q, one, None), (up, one, None), device="cuda:0")
    x = torch.zeros(1, K, dtype=torch.float16, device="cuda:0"); x[0, 0] = 100.0
    h = torch.empty(1, N, dtype=torch.float32, device="cuda:0")
    for act in ("silu", "gelu", "relu"):
        sgemv.sgemv_q4_run_gated(m.desc, m.blob, x, h, act=act)
        assert (h[0, :16] == 700.0 * 100.0).all() and (h[0, 16:] == 0).all()


@pytest.mark.parametrize("seed", range(60))
def test_random_combinations(seed):
    rng = np.random.default_rng(9000 + seed)
    pick = lambda *a: a[int(rng.integers(len(a)))]  # noqa: E731
    size = lambda lo, hi: int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))  # noqa: E731
    N, K, M, group, xt = size(1, 3000), size(1, 6000), int(rng.integers(1, 17)), pick(32, 64, 128), pick("f16", "bf16")
    zeros, bias = bool(rng.random() < 0.6), bool(rng.random() < 0.5)
    if rng.random() < 0.4:
        check_gated(9000 + seed, min(N, 1500), K, M, group, xt, pick(xt, "f32"), pick("silu", "gelu", "relu"), zeros, bias)
    else:
        check_product(9000 + seed, N, K, M, group, xt, pick(xt, "f32"), zeros, bool(rng.random() < 0.4), bias,
                      pick(None, N + int(rng.integers(1, 40))))


# ---------------------------------------------------------------------------
# streams, graphs, offsets
# ---------------------------------------------------------------------------
def test_repeats_streams_and_graph():
    """The same bits again, on another stream, and from a captured graph that
    is replayed with eager calls on other inputs in between."""
    from activation_sparse_bit_amd import sgemv
    part = problem(61, 512, 3000, 64)
    m = sgemv.Q4Matrix(*part, group=64, device="cuda:0")
    xs = [activations(62 + i, 5, 3000, "bf16").cuda() for i in range(3)]
    want = []
    for x in xs:
        y = torch.empty(5, 512, dtype=torch.bfloat16, device="cuda:0")
        sgemv.sgemv_q4_run(m.desc, m.blob, x, y)
        want.append(y)
    side = torch.cuda.Stream()
    y = torch.empty_like(want[0])
    side.wait_stream(torch.cuda.current_stream())
    sgemv.sgemv_q4_run(m.desc, m.blob, xs[0], y, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0])
    static = xs[0].clone()
    out = torch.empty_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sgemv.sgemv_q4_run(m.desc, m.blob, static, out)
    for i in (0, 1, 2, 1, 0):
        static.copy_(xs[i])
        graph.replay()
        other = torch.empty_like(out)
        sgemv.sgemv_q4_run(m.desc, m.blob, xs[(i + 1) % 3], other)
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and torch.equal(other, want[(i + 1) % 3])


def test_two_calls_at_once():
    """Calls on two streams over one matrix do not disturb each other."""
    from activation_sparse_bit_amd import sgemv
    part = problem(71, 4096, 4096, 128)
    m = sgemv.Q4Matrix(*part, device="cuda:0")
    xs = [activations(72 + i, 2, 4096, "f16").cuda() for i in range(2)]
    want = [torch.empty(2, 4096, dtype=torch.float16, device="cuda:0") for _ in xs]
    for x, y in zip(xs, want):
        sgemv.sgemv_q4_run(m.desc, m.blob, x, y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[torch.empty_like(want[0]) for _ in range(20)] for _ in xs]
    for i in range(20):
        for k in range(2):
            sgemv.sgemv_q4_run(m.desc, m.blob, xs[k], got[k][i], stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(y, want[k]) for y in got[k])


def test_offsets_beyond_32_bits():
    """Codes past 4 GiB: a blob of random codes made on the GPU, its rows
    decoded by the layout formula."""
    import ctypes
    from activation_sparse_bit_amd import sgemv
    N, K, group = 1 << 20, 9000, 128
    d = sgemv.Q4Desc()
    assert sgemv.lib().sgemv_q4_pack(None, None, None, N, K, group, 0, None, 0, ctypes.byref(d)) == 0
    assert d.w_bytes > 1 << 32
    blob = torch.empty(d.total_bytes, dtype=torch.uint8, device="cuda:0")
    gen = torch.Generator(device="cuda:0").manual_seed(1)
    for a in range(0, d.total_bytes, 1 << 30):
        blob[a:a + (1 << 30)].random_(0, 256, generator=gen)
    blob[d.s_off:d.s_off + d.s_bytes].view(torch.float16).fill_(0.01)
    x = activations(5, 2, K, "f16")
    y = torch.empty(2, N, dtype=torch.float32, device="cuda:0")
    sgemv.sgemv_q4_run(d, blob, x.cuda(), y)
    torch.cuda.synchronize()
    B = -(-K // 128)
    k = np.arange(K)
    b, j, c, i = k // 128, k // 32 % 4, k // 8 % 4, k % 8
    nibble = (i >> 1) + 4 * (i & 1)
    rows = [0, 17, N // 2 + 3, N - 16, N - 1]
    for n in rows:
        at = d.w_off + ((n // 16) * B + b) * 1024 + (16 * c + n % 16) * 16 + 4 * j + nibble // 2
        byte = blob[torch.from_numpy(at).cuda()].cpu().numpy()
        q = ((byte >> (4 * (nibble % 2))) & 15)[None, :]
        s = torch.full((1, -(-K // group)), 0.01, dtype=torch.float16)
        ref = oracle.q4_product(f64(x), q, f64(s), None, group)
        check(y[:, n:n + 1], ref, accumulation(x, (q, s, None), group) + rounding(ref, "f32"), f"row {n}")


# ---------------------------------------------------------------------------
# gates far out, infinities, sums near the end of fp32
# ---------------------------------------------------------------------------
def gates_at(values, ups, act):
    """h in fp32 for gates of exactly -7 .. 7 times `values` (a row each) and
    up projections of exactly `ups`: one code and one input each."""
    from activation_sparse_bit_amd import sgemv
    N, K = 15, 64
    gate, up = (np.full((N, K), 8, dtype=np.uint8) for _ in range(2))
    gate[:, 0], up[:, 1] = np.arange(1, 16), 9
    one = np.ones((N, 1), dtype=np.float16)
    m = sgemv.Q4Matrix.gated((gate, one, None), (up, one, None), device="cuda:0")
    x = torch.zeros(len(values), K, dtype=torch.float16)
    x[:, 0], x[:, 1] = torch.tensor(values), torch.tensor(ups)
    h = torch.empty(len(values), N, dtype=torch.float32, device="cuda:0")
    sgemv.sgemv_q4_run_gated(m.desc, m.blob, x.cuda(), h, act=act)
    return f64(x[:, :1]) * np.arange(-7, 8), f64(x[:, 1:2]), f64(h)


def test_gelu_keeps_its_relative_accuracy_far_out():
    """gelu(v) = v erfc(t) / 2, t = -v / sqrt 2 (relative to the value also
    where 1 + erf cancels).  t is off by two roundings, 2^-23 of it; erfc's
    condition number is at most 2 t^2 + 1 = v^2 + 1 (for t < 0 below 1); the
    library function within 16 steps of 2^-23 (the bound that OpenCL sets),
    two products 2^-24 each."""
    import math
    for values in (np.linspace(0.05, 1.7, 16), np.linspace(0.3, 1.0, 7)):
        g, u, h = gates_at(values, [1.0 + i / 8 for i in range(len(values))], "gelu")
        ref = np.vectorize(lambda v: 0.5 * v * math.erfc(-v * math.sqrt(0.5)))(g) * u
        check(h, ref, np.abs(ref) * (g * g + 1 + 16 + 1) * 2.0 ** -23)


def test_silu_where_the_exponential_leaves_fp32():
    """silu(v) = v e^v / (1 + e^v) below zero: e^-v is infinite from v = -88.7
    on, silu(v) u is not 0 there.  e^v within 3 steps of 2^-23 (OpenCL's
    bound) and half a subnormal, the sum, the quotient and two products 2^-24
    each, each at worst half a subnormal (2^-150) more."""
    g, u, h = gates_at([2.0, 5.0, 11.0, 12.0, 12.25, 12.5, 12.75, 13.0, 13.25, 13.5, 13.75, 14.0, 14.25],
                       [60000.0] * 11 + [1.0, 512.0], "silu")
    ref = oracle.gate_function(g, "silu") * u
    tol = np.abs(ref) * (3 + 2) * 2.0 ** -23 + (np.abs(g) + 2) * np.abs(u) * 2.0 ** -149 + 2.0 ** -149
    assert (np.abs(ref) > 3 * tol).sum() > 150   # of 195: most are far above the subnormals
    check(h, ref, tol * (1 + 2.0 ** -20))


@pytest.mark.parametrize("N,K,M,group,zeros", [(48, 260, 6, 64, True), (17, 100, 1, 128, False), (40, 1000, 3, 32, True),
                                               (8300, 384, 2, 64, True), (8300, 300, 16, 128, True), (8300, 257, 7, 32, False),
                                               (16500, 300, 16, 32, True), (33000, 384, 12, 64, True), (300, 4224, 16, 64, True),
                                               (300, 8192, 1, 128, True)])
def test_bf16_infinities_and_sums_near_the_end_of_fp32(N, K, M, group, zeros):
    """bf16 rows with an infinity give the infinity or NaN that the formula
    has, as fp16 rows do; rows of which 32 times the sum leaves fp32, but not
    the sum itself, give that sum; the other rows keep their bits."""
    part = problem(N + K, N, K, group, zeros)
    x = activations(N + M, M, K, "bf16")
    clean = run_product(x, part, group, "f32")
    kinds = ["inf", "-inf", "large", "nan", "clean", "two"] if M > 1 else ["inf", "large"]
    for turn in range(len(kinds) if M == 1 else 1):
        xs, kind = x.clone(), [kinds[(m + turn) % len(kinds)] for m in range(M)]
        for m, k in enumerate(kind):
            at = (K - 1, 7, K // 2)[m % 3]
            if k in ("inf", "-inf", "nan"):
                xs[m, at] = float(k)
            elif k == "large":
                xs[m, at] = 2e37     # times 31 beyond fp32, times 15 not
            elif k == "two":
                xs[m, at], xs[m, at - 3] = float("inf"), float("-inf")
        got = run_product(xs, part, group, "f32")
        ref = oracle.q4_product(f64(xs), part[0], f64(part[1]), part[2], group)
        finite = np.array([k in ("large", "clean") for k in kind])
        if finite.any():
            rows = np.flatnonzero(finite)
            check(got[rows], ref[rows], accumulation(xs[rows], part, group) + rounding(ref[rows], "f32") * 1.01)
        for m, k in enumerate(kind):
            if k == "clean":
                assert torch.equal(got[m], clean[m])
            elif not finite[m]:
                assert np.array_equal(f64(got[m]), ref[m], equal_nan=True), (m, k)


@pytest.mark.parametrize("N,K,M,group", [(100, 515, 4, 64), (8300, 384, 16, 64), (4200, 300, 2, 128)])
def test_gated_bf16_infinities(N, K, M, group):
    from activation_sparse_bit_amd import sgemv
    gate, up = problem(N, N, K, group), problem(N + 1, N, K, group)
    m = sgemv.Q4Matrix.gated(gate, up, group=group, device="cuda:0")
    x = activations(N + 2, M, K, "bf16") * 0.3
    run = lambda x: sgemv.sgemv_q4_run_gated(m.desc, m.blob, x.cuda(), h, act="relu")  # noqa: E731
    h = torch.empty(M, N, dtype=torch.float32, device="cuda:0")
    run(x)
    clean = h.clone()
    x[1, K - 1] = float("inf")
    run(x)
    rows = [r for r in range(M) if r != 1]
    assert torch.equal(h[rows], clean[rows])
    with np.errstate(invalid="ignore"):
        g, u = (oracle.q4_product(f64(x[1:2]), p[0], f64(p[1]), p[2], group) for p in (gate, up))
        ref = oracle.gate_function(g, "relu") * u
    assert np.array_equal(f64(h[1:2]), ref, equal_nan=True)


# ---------------------------------------------------------------------------
# kernel instances by size: streamed codes, sixteen wavefronts, pairs of both
# ---------------------------------------------------------------------------
def on_gpu(seed, N, K, group, zeros):
    gen = torch.Generator(device="cuda:0").manual_seed(seed)
    g = -(-K // group)
    q = torch.randint(0, 16, (N, K), dtype=torch.uint8, device="cuda:0", generator=gen)
    s = (0.01 + 0.01 * torch.rand(N, g, device="cuda:0", generator=gen)).half()
    z = torch.randint(0, 16, (N, g), dtype=torch.uint8, device="cuda:0", generator=gen) if zeros else None
    return q, s, z


def sampled(part, rows):
    q, s, z = part
    return q[rows].cpu().numpy(), s[rows].cpu(), None if z is None else z[rows].cpu().numpy()


def check_sampled_product(N, K, M, group, xt, zeros=True):
    from activation_sparse_bit_amd import sgemv
    part = on_gpu(N + M, N, K, group, zeros)
    m = sgemv.Q4Matrix(*part, group=group)
    x = activations(M, M, K, xt)
    y = torch.full((M + 1, N), float("nan"), dtype=torch.float32, device="cuda:0")
    sgemv.sgemv_q4_run(m.desc, m.blob, x.cuda(), y[:M])
    rows = np.array(sorted({0, 1, 15, 16, 33, 63, 64, N // 2, N // 3, N - 17, N - 2, N - 1}))
    p = sampled(part, rows)
    ref = oracle.q4_product(f64(x), p[0], f64(p[1]), p[2], group)
    check(y[:M, rows], ref, accumulation(x, p, group) + rounding(ref, "f32") * 1.01, f"N={N} K={K} M={M}")
    assert torch.isnan(y[M]).all() and torch.isfinite(y[:M]).all()
    return m


def check_sampled_gated(N, K, M, group, xt, zeros=True):
    from activation_sparse_bit_amd import sgemv
    gate, up = on_gpu(N + M, N, K, group, zeros), on_gpu(N + M + 1, N, K, group, zeros)
    m = sgemv.Q4Matrix.gated(gate, up, group=group)
    x = activations(M, M, K, xt) * 0.03
    h = torch.full((M + 1, N), float("nan"), dtype=torch.float32, device="cuda:0")
    sgemv.sgemv_q4_run_gated(m.desc, m.blob, x.cuda(), h[:M], act="relu")
    rows = np.array(sorted({0, 1, 15, 16, 31, 33, N // 2, N // 3, N - 17, N - 2, N - 1}))
    pg, pu = sampled(gate, rows), sampled(up, rows)
    g, u = (oracle.q4_product(f64(x), p[0], f64(p[1]), p[2], group) for p in (pg, pu))
    eg, eu = accumulation(x, pg, group), accumulation(x, pu, group)
    ref = oracle.gate_function(g, "relu") * u   # |relu'| <= 1, one product
    tol = eg * (np.abs(u) + eu) + np.abs(g) * eu + 2.0 ** -24 * np.abs(ref)
    check(h[:M, rows], ref, tol * (1 + 2.0 ** -7) + rounding(ref, "f32") * 1.01, f"N={N} K={K} M={M}")
    assert torch.isnan(h[M]).all() and torch.isfinite(h[:M]).all()
    return m


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
@pytest.mark.parametrize("N,M", [(8200, 3), (8200, 8), (8200, 15), (20000, 13), (7100, 2), (7100, 16)])
def test_product_streamed_every_group(N, M, xt, group):
    K = -(-(96 << 21) // N // 128) * 128 + 37
    assert check_sampled_product(N, K, M, group, xt, zeros=group != 64).desc.w_bytes >= 96 << 20


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
@pytest.mark.parametrize("N,M", [(4104, 4), (4104, 6), (4104, 16), (10000, 1), (10000, 16)])
def test_gated_streamed(N, M, xt, group):
    K = -(-(96 << 20) // N // 128) * 128 + 45
    assert check_sampled_gated(N, K, M, group, xt, zeros=group != 32).desc.w_bytes >= 96 << 20


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_sixteen_rows_on_sixteen_wavefronts(xt, group):
    """256 workgroups of one, two and four tiles over long inputs: the most
    threads and shared memory that a launch has."""
    check_sampled_product(4096, 4096, 16, group, xt)
    check_sampled_product(8192, 4096, 16, group, xt)
    check_sampled_product(16384, 4100, 16, group, xt, zeros=False)
    check_sampled_gated(4096, 4096, 16, group, xt)
    check_sampled_gated(8192, 4103, 16, group, xt)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_pairs_and_rows_of_ordinary_size(xt, group):
    """Pairs of one and two tiles each for few rows, sixteen wavefronts and
    eight."""
    for N, K, M in ((1000, 4096, 1), (1000, 4096, 8), (6000, 1000, 4), (6000, 8200, 8), (14336, 520, 2), (9000, 4096, 1)):
        check_sampled_gated(N, K, M, group, xt, zeros=M != 4)
