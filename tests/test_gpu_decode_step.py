"""The feed-forward half of a decode step and its head, the operators run
together as a decoder runs them: the attention output projection (dense input,
4-bit), the norms around the blocks, the gated 4-bit pair, the sparse down
projection over its thresholded output, the last norm and a head with an odd
number of outputs.  Every stage is checked against its definition on the very
inputs that the previous stage left, and the whole step from a captured graph
gives the eager bits."""
import numpy as np
import pytest

import oracle
import synth
from tests import gpu_util as G
from tests.test_gpu_block_norm import expected, inside
from tests.test_gpu_q4 import accumulation, check, f64, problem, rounding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D, F, V, GROUP = 1024, 2048, 5003, 64
P_SPARSE = 0.5


class Step:
    def __init__(self, M):
        from activation_sparse_bit_amd import sgemv
        self.lib, self.M, dev = sgemv, M, "cuda:0"
        self.parts = {n: problem(i, *nk, GROUP, zeros=n != "head") for i, (n, nk) in enumerate(
            {"o": (D, D), "gate": (F, D), "up": (F, D), "head": (V, D)}.items())}
        self.o = sgemv.Q4Matrix(*self.parts["o"], group=GROUP, device=dev)
        self.gu = sgemv.Q4Matrix.gated(self.parts["gate"], self.parts["up"], group=GROUP, device=dev)
        self.head = sgemv.Q4Matrix(*self.parts["head"], group=GROUP, device=dev)
        self.down_w = synth.random_int4_problem(9, D, F)
        self.down = sgemv.PackedMatrix(*self.down_w, device=dev, max_batch=M)
        rng = np.random.default_rng(10)
        t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).half().to(dev)  # noqa: E731
        self.attn, self.resid = t(M, D), t(M, D)
        self.w1, self.w2, self.post = (1 + 0.1 * t(D) for _ in range(3))
        h = lambda n, dt=torch.float16: torch.full((M, n), float("nan"), dtype=dt, device=dev)  # noqa: E731
        self.yo, self.x1, self.r1, self.hh, self.yd, self.x2, self.r2 = h(D), h(D), h(D), h(F), h(D, torch.float32), h(D), h(D)
        self.logits = h(V, torch.float32)
        self.t = [0.05] * M

    def run(self):
        s = self.lib
        s.sgemv_q4_run(self.o.desc, self.o.blob, self.attn, self.yo)
        s.sgemv_block_norm(self.x1, self.resid, self.yo, self.r1, weight=self.w1, post_weight=self.post, scale=0.5)
        s.sgemv_q4_run_gated(self.gu.desc, self.gu.blob, self.x1, self.hh, act="silu")
        s.sgemv_run_fused(self.down.desc, self.down.blob, self.hh, self.t, self.yd, self.down.workspace)
        s.sgemv_block_norm(self.x2, self.r1, self.yd, self.r2, weight=self.w2)
        s.sgemv_q4_run(self.head.desc, self.head.blob, self.x2, self.logits)

    def outputs(self):
        return self.yo, self.x1, self.r1, self.hh, self.yd, self.x2, self.r2, self.logits


@pytest.mark.parametrize("M", [1, 2, 5, 16])
def test_stages_match_their_definitions(M):
    st = Step(M)
    st.run()
    torch.cuda.synchronize()
    prod = lambda x, n: oracle.q4_product(f64(x), st.parts[n][0], f64(st.parts[n][1]), st.parts[n][2], GROUP)  # noqa: E731
    acc = lambda x, n: accumulation(x, st.parts[n], GROUP)  # noqa: E731
    ref = prod(st.attn, "o")
    check(st.yo, ref, (acc(st.attn, "o") + rounding(ref, "f16")) * 1.01, "o")
    for x, r, y, res, w, pw, scale in ((st.x1, st.r1, st.yo, st.resid, st.w1, st.post, 0.5),
                                       (st.x2, st.r2, st.yd, st.r1, st.w2, None, 1.0)):
        p = {"residual": res, "y": y, "gate": None, "weight": w, "bias": None, "post_weight": pw, "post_bias": None}
        (rr, rt), (xr, xt) = expected(p, scale, pw is not None, False, False, 1e-6, "f16", "f16")
        inside(r, rr, rt, "r"); inside(x, xr, xt, "x")
    g, u = prod(st.x1, "gate"), prod(st.x1, "up")
    ref = oracle.gate_function(g, "silu") * u
    tol = 1.13 * (acc(st.x1, "gate") + 2.0 ** -20 * np.abs(g)) * (np.abs(u) + 1) + (np.abs(g) + 1) * acc(st.x1, "up")
    check(st.hh, ref, tol + 1.02 * rounding(ref, "f16"), "gated")
    q, s, z = st.down_w
    y_ref, B, _ = oracle.gemv_masked(q, s, z, st.hh.cpu().numpy(), st.t)
    G.check_y(f64(st.yd), y_ref, B, "down")
    ref = prod(st.x2, "head")
    check(st.logits, ref, (acc(st.x2, "head") + rounding(ref, "f32")) * 1.01, "head")


def test_step_in_a_graph():
    st = Step(2)
    st.run()
    want = [t.clone() for t in st.outputs()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    for i in range(4):
        for t in st.outputs():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(st.outputs(), want))
        st.run()   # an eager step between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(st.outputs(), want))
