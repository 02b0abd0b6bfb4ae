"""The norms around a block against their float64 definition.

Tolerance.  A row sum in fp32 has at most 64 terms a lane, 6 steps over a
wavefront and 16 over the wavefronts, each off by half a step of 2^-23: a sum
of squares is off by at most 86 * 2^-24 of itself plus its own products'
2^-24, the inverse root by half of that and four roundings more, so a normed
value v^ is off by at most 50 * 2^-24 |v^|.  Subtracting a mean that is off
by 88 * 2^-24 mean|v| moves every value by that (and its square root's
argument by no more in proportion).  These go through the weight, the gate and
the residual addition with one rounding each, and through the second norm,
where an error e of the row's values moves v^ by at most
max(e) / sigma * (1 + |v^|).  The output type adds half a step."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def half_step(v, t):
    return np.abs(v) * torch.finfo(T[t]).eps / 2 + (2.0 ** -25 if t == "f16" else 2.0 ** -134)


def norm_tol(v, e, weight, bias, center, plus_one, eps):
    """Error of norm(v) when v is off by at most e."""
    dev = v - v.mean(-1, keepdims=True) if center else v
    sigma = np.sqrt((dev * dev).mean(-1, keepdims=True) + eps)
    vh = np.abs(dev) / sigma
    if center:
        e = 2 * e + 88 * U * np.abs(v).mean(-1, keepdims=True) + U * np.abs(dev)
    out = 50 * U * vh + e.max(-1, keepdims=True) / sigma * (1 + vh)
    w = np.ones(v.shape[-1]) if weight is None else np.abs(weight + (1.0 if plus_one else 0.0))
    out = out * w + 2 * U * vh * w
    return out if bias is None else out + U * (vh * w + np.abs(bias))


def make(seed, rows, D, r, y, x, w, post, gate, center, plus_one, bias, offset=0.3, device="cuda:0"):
    rng = np.random.default_rng(seed)
    t = lambda a, k: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(T[k]).to(device)  # noqa: E731
    p = {"residual": t(2 * rng.standard_normal((rows, D)) + offset, r),
         "y": None if y is None else t(rng.standard_normal((rows, D)) - offset, y)}
    c = 0.0 if plus_one else 1.0
    p["weight"] = t(c + 0.2 * rng.standard_normal(D), w) if w else None
    p["bias"] = t(rng.standard_normal(D), w) if w and bias else None
    p["post_weight"] = t(c + 0.2 * rng.standard_normal(D), w) if w and post else None
    p["post_bias"] = t(rng.standard_normal(D), w) if w and post and bias else None
    p["gate"] = None if gate is None else t(rng.random((rows, D) if gate == "rows" else D), y)
    return p


def expected(p, scale, post, center, plus_one, eps, rt, xt):
    q = {k: f64(v) for k, v in p.items()}
    r, x = oracle.block_norm(q["residual"], q["y"], q["gate"], scale, post, q["post_weight"], q["post_bias"],
                             q["weight"], q["bias"], center, plus_one, eps)
    e = np.zeros_like(r)
    if q["y"] is not None:
        u = q["y"]
        eu = np.zeros_like(u)
        if post:
            eu = norm_tol(u, eu, q["post_weight"], q["post_bias"], center, plus_one, eps)
            u = oracle.norm(u, q["post_weight"], q["post_bias"], center, plus_one, eps)
        g = 1.0 if q["gate"] is None else q["gate"]
        e = np.abs(scale * g) * (eu + 2 * U * np.abs(u)) + 2 * U * (np.abs(r) + np.abs(q["residual"]))
    ex = norm_tol(r, e, q["weight"], q["bias"], center, plus_one, eps)
    return (r, (e + half_step(r, rt)) * 1.01), (x, (ex + half_step(x, xt)) * 1.01)


def inside(got, ref, tol, what):
    got = f64(got)
    assert np.all(np.isfinite(got)), f"{what}: non-finite"
    over = np.abs(got - ref) - tol
    assert not (over > 0).any(), f"{what}: {int((over > 0).sum())} of {got.size} outside, worst by {over.max():.3e}"


def check(seed, rows, D, r="f16", y="f16", x="f16", w="f16", post=False, gate=None, scale=1.0, center=False,
          plus_one=False, bias=False, eps=1e-5, r_out=True):
    from activation_sparse_bit_amd import sgemv
    p = make(seed, rows, D, r, y, x, w, post, gate, center, plus_one, bias)
    xo = torch.full((rows + 1, D), float("nan"), dtype=T[x], device="cuda:0")
    ro = torch.full((rows + 1, D), float("nan"), dtype=T[r], device="cuda:0")
    kept = {k: None if v is None else v.clone() for k, v in p.items()}
    sgemv.sgemv_block_norm(xo[:rows], p["residual"], p["y"], ro[:rows] if r_out else None, weight=p["weight"], bias=p["bias"],
                           post_weight=p["post_weight"], post_bias=p["post_bias"], gate=p["gate"], scale=scale, eps=eps,
                           post_norm=post, center=center, plus_one=plus_one)
    torch.cuda.synchronize()
    (rr, rtol), (xr, xtol) = expected(p, scale, post, center, plus_one, eps, r, x)
    if r_out:
        inside(ro[:rows], rr, rtol, "residual_out")
    inside(xo[:rows], xr, xtol, "x")
    assert torch.isnan(xo[rows]).all() and torch.isnan(ro[rows if r_out else 0:]).all()
    for k, v in p.items():
        assert v is None or torch.equal(v, kept[k]), k


@pytest.mark.parametrize("D", [1, 2, 7, 8, 9, 63, 64, 65, 511, 512, 513, 1000, 2047, 2048, 2049, 4096, 4097, 5001, 8192,
                               8200, 12345, 16384, 16385, 28672, 32768, 32769, 65535, 65536])
@pytest.mark.parametrize("center", [False, True])
def test_widths(D, center):
    rows = 1 if D % 2 else 5
    check(D, rows, D, post=True, gate="vector" if D % 3 else "rows", scale=0.5, center=center, bias=True)


@pytest.mark.parametrize("r,y,x,w", [(r, y, x, w) for r in T for y in T for x in T for w in T])
def test_types(r, y, x, w):
    check(7, 3, 300, r, y, x, w, post=True, gate="rows", scale=0.22, center=True, plus_one=True, bias=True)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "vector", "rows"])
@pytest.mark.parametrize("plus_one", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_combinations(post, gate, plus_one, bias):
    check(13, 9, 1234, "f32", "bf16", "bf16", "f32", post, gate, 0.7, False, plus_one, bias)


def test_without_block_output_and_weights():
    check(17, 4, 777, y=None, w=None)
    check(18, 4, 4096, y=None, r_out=False, r="f32", x="bf16", center=True)
    check(19, 4, 700, w=None, post=True)


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 257, 5000])
def test_row_counts(rows):
    check(rows, rows, 96, "bf16", "bf16", "bf16", "bf16", post=True)
    check(rows, rows, 640, "f16", "f32", "f16", "f16")


@pytest.mark.parametrize("rows,D", [(513, 1032), (600, 1100), (700, 4099), (520, 8193), (300, 9000), (260, 16390),
                                    (257, 12288), (512, 8200), (20, 20001), (9, 33000), (600, 8191)])
@pytest.mark.parametrize("center", [False, True])
def test_many_rows_and_widths(rows, D, center):
    """Every number of runs a thread has, with and without odd elements."""
    check(rows + D, rows, D, "bf16", "f32" if D % 2 else "bf16", "bf16", "f32", post=True, gate="rows", scale=0.5,
          center=center, bias=True)


@pytest.mark.parametrize("seed", range(80))
def test_random_combinations(seed):
    rng = np.random.default_rng(7000 + seed)
    pick = lambda *a: a[int(rng.integers(len(a)))]  # noqa: E731
    size = lambda lo, hi: int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))  # noqa: E731
    D = size(1, 40000)
    rows = size(1, max(2, min(1500, (1 << 21) // D)))
    y = pick("f16", "bf16", "f32", None)
    flag = lambda p: bool(rng.random() < p)  # noqa: E731
    check(7000 + seed, rows, D, pick(*T), y, pick(*T), pick("f16", "bf16", "f32", None), post=y is not None and flag(0.5),
          gate=None if y is None else pick(None, "vector", "rows"), scale=pick(1.0, 0.5, -0.3), center=flag(0.4),
          plus_one=flag(0.3), bias=flag(0.5), eps=pick(1e-5, 1e-3), r_out=flag(0.8))


@pytest.mark.parametrize("D", [8, 11])
def test_more_rows_than_a_launch_takes(D):
    """More than 2^21 rows: two launches; the last rows as one call has them."""
    from activation_sparse_bit_amd import sgemv
    rows, n = (1 << 21) + 6, 9
    gen = torch.Generator(device="cuda:0").manual_seed(D)
    r = torch.randn(rows, D, device="cuda:0", generator=gen).half()
    y = torch.randn(rows, D, device="cuda:0", generator=gen).bfloat16()
    gate = torch.rand(rows, D, device="cuda:0", generator=gen).bfloat16()
    x, ro = torch.full((rows + 1, D), 7.0, device="cuda:0"), torch.empty_like(r)
    sgemv.sgemv_block_norm(x[:rows], r, y, ro, gate=gate, post_norm=True)
    for a, b in ((0, n), ((1 << 21) - 4, (1 << 21) + 6)):
        want, want_r = torch.empty(b - a, D, device="cuda:0"), torch.empty(b - a, D, device="cuda:0").half()
        sgemv.sgemv_block_norm(want, r[a:b], y[a:b], want_r, gate=gate[a:b], post_norm=True)
        torch.cuda.synchronize()
        assert torch.equal(x[a:b], want) and torch.equal(ro[a:b], want_r)
    assert (x[rows] == 7).all()


def test_expanded_gate():
    from activation_sparse_bit_amd import sgemv
    p = make(3, 5, 200, "f16", "f16", "f16", "f16", False, "vector", False, False, False)
    out = [torch.empty_like(p["residual"]) for _ in range(2)]
    for x, g in zip(out, (p["gate"], p["gate"].expand(5, 200))):
        sgemv.sgemv_block_norm(x, p["residual"], p["y"], weight=p["weight"], gate=g)
    torch.cuda.synchronize()
    assert torch.equal(*out)


def test_no_rows():
    from activation_sparse_bit_amd import sgemv
    x, r = torch.empty(0, 64, device="cuda:0"), torch.empty(0, 64, device="cuda:0")
    sgemv.sgemv_block_norm(x, r, r, r)


def test_in_place_and_strided():
    """residual_out in residual's place, x in y's, both as columns of one
    wider buffer that starts off a 16-byte boundary."""
    from activation_sparse_bit_amd import sgemv
    rows, D = 6, 1001
    p = make(3, rows, D, "bf16", "bf16", "bf16", "f32", True, "rows", False, False, False)
    (rr, rtol), (xr, xtol) = expected(p, 0.5, True, False, False, 1e-6, "bf16", "bf16")
    wide = torch.full((rows, 2 * D + 7), 9.0, dtype=torch.bfloat16, device="cuda:0")
    a, b = wide[:, 3:3 + D], wide[:, 5 + D:5 + 2 * D]
    a.copy_(p["residual"]); b.copy_(p["y"])
    sgemv.sgemv_block_norm(b, a, b, a, weight=p["weight"], post_weight=p["post_weight"], gate=p["gate"], scale=0.5)
    torch.cuda.synchronize()
    inside(a, rr, rtol, "residual_out"); inside(b, xr, xtol, "x")
    left = torch.ones(2 * D + 7, dtype=torch.bool)
    left[3:3 + D] = False; left[5 + D:5 + 2 * D] = False
    assert (wide[:, left.cuda()] == 9).all()


def test_unrounded_between_norms():
    """x is the norm of r before r is rounded: a residual of 256 in bf16
    swallows y, its norm does not."""
    from activation_sparse_bit_amd import sgemv
    r = torch.full((1, 64), 256.0, dtype=torch.bfloat16, device="cuda:0")
    y = torch.zeros_like(r); y[0, 0] = 0.5
    x = torch.empty(1, 64, device="cuda:0")
    sgemv.sgemv_block_norm(x, r, y, r, center=True, eps=0.0)
    assert (r == 256).all()
    ref = oracle.norm(256.0 + f64(y), center=True)
    assert np.allclose(f64(x), ref, rtol=1e-4)


def test_non_finite_rows_stay_apart():
    from activation_sparse_bit_amd import sgemv
    p = make(23, 6, 500, "f16", "f16", "f16", "f16", True, None, False, False, False)
    x, ro = torch.empty_like(p["residual"]), torch.empty_like(p["residual"])
    run = lambda: sgemv.sgemv_block_norm(x, p["residual"], p["y"], ro, weight=p["weight"], post_weight=p["post_weight"])  # noqa: E731
    run()
    x0, r0 = x.clone(), ro.clone()
    p["y"][2, 499], p["residual"][4, 0] = float("nan"), float("inf")
    run()
    for m in (0, 1, 3, 5):
        assert torch.equal(x[m], x0[m]) and torch.equal(ro[m], r0[m])
    assert torch.isnan(x[2]).all() and torch.isnan(ro[2]).all()
    assert torch.isinf(ro[4, 0]) and torch.equal(ro[4, 1:], r0[4, 1:]) and torch.isnan(x[4, 0]) and (x[4, 1:] == 0).all()


def test_zero_rows_with_eps():
    from activation_sparse_bit_amd import sgemv
    r = torch.zeros(3, 200, device="cuda:0")
    x = torch.empty_like(r)
    sgemv.sgemv_block_norm(x, r, r.clone(), post_norm=True, center=True)
    assert (x == 0).all()


def test_streams_and_graph():
    from activation_sparse_bit_amd import sgemv
    p = make(29, 16, 4096, "f32", "bf16", "bf16", "bf16", True, "vector", False, True, False)
    x, ro = torch.empty_like(p["y"]), torch.empty_like(p["residual"])
    kw = dict(weight=p["weight"], post_weight=p["post_weight"], gate=p["gate"], scale=0.5, plus_one=True)
    sgemv.sgemv_block_norm(x, p["residual"], p["y"], ro, **kw)
    x0, r0 = x.clone(), ro.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x.zero_(); side.wait_stream(torch.cuda.current_stream())
    sgemv.sgemv_block_norm(x, p["residual"], p["y"], ro, stream=side, **kw)
    side.synchronize()
    assert torch.equal(x, x0) and torch.equal(ro, r0)
    res, y = p["residual"].clone(), p["y"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sgemv.sgemv_block_norm(x, res, y, res, **kw)   # the residual in place
    for i in range(4):
        res.copy_(p["residual"])
        graph.replay()
        sgemv.sgemv_block_norm(torch.empty_like(x), r0, p["y"], **kw)
        torch.cuda.synchronize()
        assert torch.equal(x, x0) and torch.equal(res, r0)


def test_wide_strides_beyond_32_bits():
    """Two fp32 rows 8 GiB apart."""
    from activation_sparse_bit_amd import sgemv
    D, ld = 512, (1 << 31) - 8
    big = torch.empty(ld + D, dtype=torch.float32, device="cuda:0")
    rows = big.as_strided((2, D), (ld, 1))
    p = make(31, 2, D, "f32", "f16", "f16", "f16", False, None, False, False, False)
    rows.copy_(p["residual"])
    x, ro = torch.empty_like(p["y"]), torch.empty_like(p["residual"])
    sgemv.sgemv_block_norm(x, rows, p["y"], rows, weight=p["weight"])
    want_x, want_r = torch.empty_like(x), torch.empty_like(ro)
    sgemv.sgemv_block_norm(want_x, p["residual"], p["y"], want_r, weight=p["weight"])
    torch.cuda.synchronize()
    assert torch.equal(x, want_x) and torch.equal(rows.contiguous(), want_r)


# widths of every number of runs a thread has for few rows (a wavefront a row, 1, 2, 4, 8 runs), with and without odd elements
WIDTHS = [304, 307, 1000, 4099, 12000, 12003, 20000, 20001, 33000, 33001]


@pytest.mark.parametrize("r,y", [(r, y) for r in T for y in T])
@pytest.mark.parametrize("D", WIDTHS)
def test_types_at_every_width(D, r, y):
    """Both norms, a gate a row; x and the vectors take each type in turn."""
    i = WIDTHS.index(D) + 3 * list(T).index(r) + list(T).index(y)
    x, w = list(T)[i % 3], list(T)[(i // 3) % 3]
    check(D + i, 3, D, r, y, x, w, post=True, gate="rows", scale=0.5, center=i % 2 == 0, plus_one=i % 4 == 0, bias=i % 3 == 0)


@pytest.mark.parametrize("rows,D", [(300, 8200), (300, 8201), (260, 12003), (257, 16385), (600, 4104), (600, 4097)])
@pytest.mark.parametrize("r,y", [("f32", "bf16"), ("f32", "f32"), ("f16", "f32"), ("bf16", "bf16")])
def test_types_of_many_rows(rows, D, r, y):
    check(rows + D, rows, D, r, y, "bf16", "f32", post=True, gate="rows", scale=0.5, bias=True)


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("r", list(T))
def test_without_block_output_at_every_width(D, r):
    """The norm before a model's first block."""
    check(D, 5, D, r, None, "bf16", "f16", center=D % 3 == 0, r_out=D % 2 == 0)


@pytest.mark.parametrize("rows,D", [(3, D) for D in WIDTHS] + [(300, 8200), (300, 8203), (600, 4099), (257, 16400)])
@pytest.mark.parametrize("gate", [None, "rows"])
def test_in_place_at_every_width(rows, D, gate):
    """x in y's place and residual_out in residual's, the two crossed, and x
    in the gate's place: the bits of the call with buffers of its own."""
    from activation_sparse_bit_amd import sgemv
    p = make(rows + D, rows, D, "bf16", "bf16", "bf16", "f32", True, gate, True, False, True)
    kw = dict(weight=p["weight"], bias=p["bias"], post_weight=p["post_weight"], post_bias=p["post_bias"], scale=0.5, center=True)
    want_x, want_r = torch.empty_like(p["y"]), torch.empty_like(p["y"])
    sgemv.sgemv_block_norm(want_x, p["residual"], p["y"], want_r, gate=p["gate"], **kw)
    for where in ("own", "crossed") + (("gate",) if gate else ()):
        res, y = p["residual"].clone(), p["y"].clone()
        g = None if gate is None else p["gate"].clone()
        x, ro = {"own": (y, res), "crossed": (res, y), "gate": (g, res)}[where]
        sgemv.sgemv_block_norm(x, res, y, ro, gate=g, **kw)
        torch.cuda.synchronize()
        assert torch.equal(x, want_x) and torch.equal(ro, want_r), where
