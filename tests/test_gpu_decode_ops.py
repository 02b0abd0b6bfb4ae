"""Beam search over a paged cache, the operators run together as a decoder runs
them: pages are forked for the beams that go on and grow by a token, every
layer projects (4-bit), turns queries and keys by their positions and writes
keys and values into the cache, attends over it, projects back and adds to the
residual; the head's logits choose the next beams.  Every stage is checked
against its definition on the very inputs that the previous stage left, the
cache against a history kept apart for every beam, and the whole step on
another stream and from a captured graph gives the same bits.

Tolerance.  A turned pair is off by half a step of fp16 (2^-11 of its size, or
2^-25) and by the sine's, cosine's and products' fp32 roundings, under 2^-18 of
the pair's length at these positions.  Keys and values in 8 bits are off from
the fp16 ones by half a step of e4m3 (2^-4 of their size, or 2^-10) and by the
fp16 ones' own half step.  Attention and beams are as in their own files."""
import numpy as np
import pytest

import oracle
from tests import test_gpu_beam
from tests.test_gpu_q4 import problem

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
B, W, D, HQ, HKV, DIM, V, PAGE, WIDTH, LAYERS, GROUP, END = 2, 3, 256, 4, 2, 64, 1003, 4, 6, 2, 64, 7
R, STEPS = B * W, 14
U = 2.0 ** -24


def f64(t):
    return t.detach().to(torch.float32).double().cpu().numpy()


class Decoder:
    def __init__(self, cache):
        from activation_sparse_bit_amd import sgemv as s
        self.s, self.cache_type = s, cache
        m = lambda seed, n, k: s.Q4Matrix(*problem(seed, n, k, GROUP, zeros=True), group=GROUP, device=DEV)  # noqa: E731
        self.qkv = [m(2 * i, (HQ + 2 * HKV) * DIM, D) for i in range(LAYERS)]
        self.o = [m(2 * i + 1, D, HQ * DIM) for i in range(LAYERS)]
        self.head = m(50, V, D)
        rng = np.random.default_rng(51)
        t = lambda *n: torch.from_numpy(rng.standard_normal(n).astype(np.float32)).half().to(DEV)  # noqa: E731
        self.embed, self.norm = t(V, D), [1 + 0.1 * t(D) for _ in range(LAYERS + 1)]
        self.inv_freq = (100.0 ** -(torch.arange(DIM // 2) / (DIM / 2))).to(DEV)
        pages = R * WIDTH + 3
        dtype = {"f16": torch.float16, "e4m3": torch.float8_e4m3fn}[cache]
        self.pools = [[torch.full((pages, PAGE, HKV, DIM), float("nan")).to(dtype).to(DEV) for _ in range(2)] for _ in range(LAYERS)]
        self.caches = [s.KVCache(k, v) for k, v in self.pools]
        i = lambda *n: torch.zeros(*n, dtype=torch.int32, device=DEV)  # noqa: E731
        f = lambda *n, dt=torch.float16: torch.zeros(*n, dtype=dt, device=DEV)  # noqa: E731
        self.table, self.lengths, self.refs, self.parents, self.ones = i(R, WIDTH), i(R), i(pages), i(R), i(R) + 1
        self.slots, self.pairs, self.count, self.status, self.positions = i(R, 1), i(R, 3), i(1), i(2), i(R)
        self.base = (torch.arange(R, dtype=torch.int32) // W * W).to(DEV).view(B, W)
        self.tokens, self.chosen, self.from_beam = i(B, W), i(B, W), i(B, W)
        self.scores, self.scores_out = f(B, W, dt=torch.float32), f(B, W, dt=torch.float32)
        self.finished = torch.zeros(B, W, dtype=torch.uint8, device=DEV)
        self.resid, self.x, self.y = f(R, D), f(R, D), f(R, D)
        self.projected = [f(R, (HQ + 2 * HKV) * DIM) for _ in range(LAYERS)]
        self.turned = [(f(R, HQ, DIM), f(R, HKV, DIM)) for _ in range(LAYERS)]
        self.attended = [f(R, HQ, DIM) for _ in range(LAYERS)]
        self.logits = f(R, V, dt=torch.float32)
        z = lambda n: torch.zeros(n, dtype=torch.uint8, device=DEV)  # noqa: E731
        self.ws_pages = z(s.sgemv_pages_workspace_bytes(R, WIDTH, pages))
        self.ws_attn = z(s.sgemv_attn_workspace_bytes(R, HQ, HKV, DIM))
        self.ws_beam = z(s.sgemv_beam_workspace_bytes(B, W, V, W))
        self.reset()

    def reset(self):
        for t in (self.table, self.lengths, self.refs, self.finished):
            t.zero_()
        self.parents.copy_(torch.arange(R, dtype=torch.int32))
        self.tokens.copy_(torch.tensor([[5] * W, [900] * W], dtype=torch.int32))
        self.scores.fill_(float("-inf"))
        self.scores[:, 0] = 0   # all beams are alike at first: one of them has candidates

    def pages(self):
        self.s.sgemv_pages_fork(self.table, self.lengths, self.refs, self.table, self.lengths, self.refs, self.ws_pages,
                                page_size=PAGE, pairs=self.pairs, count=self.count, status=self.status, parents=self.parents,
                                grow=self.ones, slots=self.slots, caches=self.caches)

    def layers(self):
        s = self.s
        torch.sub(self.lengths, self.ones, out=self.positions)
        self.resid.copy_(self.embed[self.tokens.view(-1).long()])
        s.sgemv_block_norm(self.x, self.resid, weight=self.norm[0])
        for i in range(LAYERS):
            s.sgemv_q4_run(self.qkv[i].desc, self.qkv[i].blob, self.x, self.projected[i])
            heads = self.projected[i].view(R, HQ + 2 * HKV, DIM)
            q, k, v = heads[:, :HQ], heads[:, HQ:HQ + HKV], heads[:, HQ + HKV:]
            s.sgemv_rotary(q, self.turned[i][0], self.positions, self.inv_freq, k=k, k_out=self.turned[i][1], v=v,
                           cache=self.caches[i], slots=self.slots.view(-1))
            s.sgemv_attn_paged(self.turned[i][0], self.caches[i], self.table, self.lengths, self.attended[i], self.ws_attn)
            s.sgemv_q4_run(self.o[i].desc, self.o[i].blob, self.attended[i].view(R, HQ * DIM), self.y)
            s.sgemv_block_norm(self.x, self.resid, self.y, self.resid, weight=self.norm[i + 1])
        s.sgemv_q4_run(self.head.desc, self.head.blob, self.x, self.logits)

    def select(self):
        self.s.sgemv_beam_select(self.logits.view(B, W, V), self.scores, self.chosen, self.from_beam, self.scores_out,
                                 self.ws_beam, finished=self.finished, end_token=END)

    def advance(self):
        self.finished.copy_(self.finished.gather(1, self.from_beam.long()) | (self.chosen == END))
        self.tokens.copy_(self.chosen)
        self.scores.copy_(self.scores_out)
        self.parents.copy_((self.from_beam + self.base).view(-1))

    def step(self):
        self.pages()
        self.layers()
        self.select()
        self.advance()

    def state(self):
        return [t.clone() for t in (self.table, self.lengths, self.refs, self.parents, self.tokens, self.scores, self.finished,
                                    self.slots, self.logits, *self.attended, *(t for pair in self.turned for t in pair))]


def attention(q, k, v):
    out, _, z = oracle.attention(q, k, v, DIM ** -0.5)
    tol = np.zeros_like(out)
    for h in range(HQ):
        g = h * HKV // HQ
        e = ((DIM + 4) * U * DIM ** -0.5 * (np.abs(k[:, g]) @ np.abs(q[h]))).max() + 8 * U * np.abs(z[h]).max()
        p = np.exp(z[h] - z[h].max())
        tol[h] = (2.0 ** -11 + 2 * e + 2.0 ** -22 + 4 * (len(k) / 128 + 64) * U) * (p @ np.abs(v[:, g]) / p.sum()) \
            + np.abs(out[h]) * 2.0 ** -11 + 2.0 ** -24
    return out, 1.01 * tol


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_stages_match_their_definitions(cache):
    d = Decoder(cache)
    history = [[[] for _ in range(R)] for _ in range(LAYERS)]
    shared = 0
    for step in range(STEPS):
        want = oracle.pages_fork(*(t.cpu().numpy() for t in (d.table, d.lengths, d.refs)), PAGE, d.parents.tolist(), [1] * R, 1)
        d.pages()
        for name, t in {"table": d.table, "lengths": d.lengths, "refs": d.refs, "slots": d.slots, "pairs": d.pairs}.items():
            assert np.array_equal(t.cpu().numpy(), want[name]), (step, name)
        assert d.status.tolist() == [0, 0]
        shared += want["count"]
        d.layers()
        for i in range(LAYERS):
            history[i] = [list(history[i][p]) for p in d.parents.tolist()]
            heads = f64(d.projected[i]).reshape(R, HQ + 2 * HKV, DIM)
            for x, got in ((heads[:, :HQ], d.turned[i][0]), (heads[:, HQ:HQ + HKV], d.turned[i][1])):
                ref = oracle.rotary(x, d.positions.cpu().numpy()[None], f64(d.inv_freq))
                size = np.concatenate([np.hypot(x[..., :DIM // 2], x[..., DIM // 2:])] * 2, axis=-1)
                assert (np.abs(f64(got) - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -18 * size).all(), (step, i)
            for r in range(R):
                history[i][r].append((f64(d.turned[i][1][r]), heads[r, HQ + HKV:]))
                held = [oracle.paged(f64(p), d.table[r].tolist(), step + 1) for p in d.pools[i]]
                for c, kept in zip(held, (np.stack(x) for x in zip(*history[i][r]))):
                    room = 0 if cache == "f16" else np.abs(kept) * (2.0 ** -4 + 2.0 ** -10) + 2.0 ** -10 + 2.0 ** -24
                    assert (np.abs(c - kept) <= room).all(), (step, i, r)
                ref, tol = attention(f64(d.turned[i][0][r]), *held)
                assert (np.abs(f64(d.attended[i][r]) - ref) <= tol).all(), (step, i, r)
        d.select()
        args = d.logits.view(B, W, V), d.scores.clone(), W, d.finished.clone(), END
        test_gpu_beam.check(*args)
        assert all(torch.equal(a, b) for a, b in zip((d.chosen, d.from_beam, d.scores_out), test_gpu_beam.run(*args)))
        d.advance()
        torch.cuda.synchronize()
    assert shared > 0 and (d.lengths == STEPS).all()   # pages were shared and copied on the way


def test_step_on_another_stream_and_in_a_graph():
    d = Decoder("f16")
    want = []
    for _ in range(STEPS):
        d.step()
        want.append(d.state())
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    d.reset()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for ref in want:
            d.step()
            assert all(torch.equal(a, b) for a, b in zip(d.state(), ref))
    stream.synchronize()
    d.reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.step()
    for n, ref in enumerate(want):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(d.state(), ref)), n


def test_two_searches_at_once():
    """Two decoders with workspaces of their own on two streams, their steps in turn."""
    a, b = Decoder("f16"), Decoder("e4m3")
    want = []
    for d in (a, b):
        for _ in range(STEPS):
            d.step()
        want.append(d.state())
        d.reset()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(STEPS):
        for d, stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                d.step()
    torch.cuda.synchronize()
    for d, ref in zip((a, b), want):
        assert all(torch.equal(x, y) for x, y in zip(d.state(), ref))


def test_one_workspace_for_all():
    """The calls of a step take turns in one workspace, which each leaves fit for the next."""
    d = Decoder("f16")
    want = []
    for _ in range(STEPS):
        d.step()
        want.append(d.state())
    d.reset()
    d.ws_pages = d.ws_attn = d.ws_beam = max((d.ws_pages, d.ws_attn, d.ws_beam), key=lambda t: t.numel())
    moved, count = torch.zeros(len(d.refs), 3, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    scratch = d.table.clone(), d.refs.clone()
    for n, ref in enumerate(want):
        d.step()
        assert all(torch.equal(a, b) for a, b in zip(d.state(), ref)), n
        d.s.sgemv_pages_compact(d.table, d.lengths, d.refs, *scratch, d.ws_pages, page_size=PAGE, pairs=moved, count=count)
    assert int(d.ws_attn[:1 << 18].count_nonzero()) == 0
