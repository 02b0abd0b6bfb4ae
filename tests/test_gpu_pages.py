"""A cache's pages: forks, growth, ends, compaction and copies, against their
row-by-row definition.  Whole numbers and copies are equal."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
T = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


class Pool:
    """A consistent state: rows of random lengths, some of which share the
    first pages of another row, and random free pages between."""

    def __init__(self, seed, rows, width, page, spare=None, heads=2, dim=16, layers=2, x="f16", layout="tokens",
                 share=0.4, empty=0.2):
        from activation_sparse_bit_amd import sgemv
        self.lib, rng = sgemv, np.random.default_rng(seed)
        lists, lengths = [], []
        taken = 0
        for r in range(rows):
            n = 0 if rng.random() < empty else int(rng.integers(1, (width - 2) * page + 1)) if width > 2 else int(rng.integers(0, page + 1))
            held = -(-n // page)
            mine = []
            if r and rng.random() < share:   # as far as a row before this one goes
                other = int(rng.integers(r))
                mine = lists[other][:held]
                if len(mine) == held and held and rng.random() < 0.5:
                    n = min(n, lengths[other]) or 0
                    held = -(-n // page)
                    mine = mine[:held]
            while len(mine) < held:
                mine = mine + [taken]
                taken += 1
            lists.append(mine)
            lengths.append(n)
        pages = taken + (rows * 3 + 5 if spare is None else spare)
        ids = rng.permutation(pages)
        table = np.full((rows, width), -7, dtype=np.int32)
        refs = np.zeros(pages, dtype=np.int32)
        for r, mine in enumerate(lists):
            table[r, :len(mine)] = ids[mine]
            for i in mine:
                refs[ids[i]] += 1
        self.table, self.lengths, self.refs, self.page, self.pages = table, np.array(lengths, dtype=np.int32), refs, page, pages
        g = torch.Generator().manual_seed(seed)
        inner = (heads, page, dim) if layout == "heads" else (page, heads, dim)
        turn = (lambda p: p.transpose(1, 2)) if layout == "heads" else (lambda p: p)
        self.kv = [tuple(turn(torch.randn(pages, *inner, generator=g).to(T[x]).to(DEV)) for _ in range(2)) for _ in range(layers)]
        self.caches = [sgemv.KVCache(k, v) for k, v in self.kv]
        self.workspace = torch.zeros(sgemv.sgemv_pages_workspace_bytes(rows, width, pages), dtype=torch.uint8, device=DEV)
        self.rng = rng

    def dev(self, *arrays):
        return [None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV) for a in arrays]

    def snapshot(self):
        return [(k.clone(), v.clone()) for k, v in self.kv]

    def check_copies(self, before, pairs):
        for (k, v), (k0, v0) in zip(self.kv, before):
            for now, was in ((k, k0), (v, v0)):
                want = was.clone()
                for s, t, n in pairs:
                    want[t, :n] = was[s, :n]
                assert torch.equal(now.view(torch.uint8) if now.is_contiguous() else now.float(),
                                   want.view(torch.uint8) if want.is_contiguous() else want.float())

    def fork(self, parents=None, grow=None, max_grow=None, in_place=False, apply=True, run=None):
        rows, width = self.table.shape
        max_grow = int(max(grow, default=0)) if max_grow is None and grow is not None else max_grow or 0
        want = oracle.pages_fork(self.table, self.lengths, self.refs, self.page, parents, grow, max_grow)
        t, n, r, p, g = self.dev(self.table, self.lengths, self.refs, parents, grow)
        kept = [x.clone() for x in (t, n, r)]
        outs = (t, n, r) if in_place else tuple(torch.full_like(x, 99) for x in (t, n, r))
        e = lambda *s: torch.full(s, 99, dtype=torch.int32, device=DEV)  # noqa: E731
        slots, pairs, count, status = e(rows, max_grow), e(rows, 3), e(1), e(2)
        before = self.snapshot()
        (run or (lambda f: f()))(lambda: self.lib.sgemv_pages_fork(
            t, n, r, *outs, self.workspace, page_size=self.page, parents=p, grow=g, slots=slots, pairs=pairs, count=count,
            status=status, caches=self.caches))
        torch.cuda.synchronize()
        got = {"table": outs[0], "lengths": outs[1], "refs": outs[2], "slots": slots, "pairs": pairs}
        assert tuple(status.tolist()) == want["status"], (status.tolist(), want["status"])
        for name, x in got.items():
            assert np.array_equal(x.cpu().numpy(), want[name]), (name, x.cpu().numpy(), want[name])
        assert count.item() == want["count"]
        if not in_place:
            assert all(torch.equal(a, b) for a, b in zip((t, n, r), kept))
        self.check_copies(before, want["pairs"][:want["count"]].tolist())
        assert int(self.workspace[:256].count_nonzero()) == 0
        if apply:
            self.table, self.lengths, self.refs = (x.cpu().numpy() for x in outs)
        return want

    def compact(self, in_place=False):
        rows, width = self.table.shape
        want = oracle.pages_compact(self.table, self.lengths, self.refs, self.page)
        t, n, r = self.dev(self.table, self.lengths, self.refs)
        outs = (t, r) if in_place else (torch.full_like(t, 99), torch.full_like(r, 99))
        pairs, count = torch.full((self.pages, 3), 99, dtype=torch.int32, device=DEV), torch.full((1,), 99, dtype=torch.int32, device=DEV)
        before = self.snapshot()
        self.lib.sgemv_pages_compact(t, n, r, *outs, self.workspace, page_size=self.page, pairs=pairs, count=count, caches=self.caches)
        torch.cuda.synchronize()
        for name, x in {"table": outs[0], "refs": outs[1], "pairs": pairs}.items():
            assert np.array_equal(x.cpu().numpy(), want[name]), name
        assert count.item() == want["count"]
        self.check_copies(before, want["pairs"][:want["count"]].tolist())
        self.table, self.refs = (x.cpu().numpy() for x in outs)


@pytest.mark.parametrize("rows,width,page", [(1, 1, 1), (1, 4, 16), (3, 6, 5), (8, 20, 16), (70, 9, 7), (256, 12, 32),
                                             (257, 12, 3), (1000, 5, 16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_random_forks(rows, width, page, in_place):
    p = Pool(rows + page, rows, width, page)
    for step in range(6):
        parents = p.rng.integers(-1, rows, rows) if step % 3 else None
        grow = p.rng.integers(0, 4, rows) if step != 2 else None
        p.fork(parents, grow, in_place=in_place)
        if p.table.shape[1] > 2:
            assert (p.refs >= 0).all()


def test_beams_change_places_and_share():
    """All rows from one: the last page is shared by all, the highest row keeps
    it; where one of them does not grow, all that do copy."""
    p = Pool(1, 6, 8, 16, empty=0, share=0)
    p.lengths[2] = 37
    p.refs[:] = 0
    for r in range(6):
        held = -(-int(p.lengths[r]) // 16)
        p.table[r, held:] = -7
        for i in p.table[r, :held]:
            p.refs[i] += 1
    want = p.fork([2] * 6, [1] * 6)
    assert want["count"] == 5 and p.table[5, 2] != p.table[4, 2]
    p.fork([0] * 6, [1, 0, 1, 2, 1, 1])
    p.fork([5, 4, 3, 2, 1, 0], [1] * 6)          # all change places
    p.fork([-1] * 6)                             # all end
    assert (p.refs == 0).all() and (p.lengths == 0).all()
    p.fork(None, [40, 0, 16, 1, 5, 3])           # begin anew


def test_out_of_pages_and_tables():
    p = Pool(2, 5, 6, 4, spare=3, empty=0)
    state = p.table.copy(), p.lengths.copy(), p.refs.copy()
    want = p.fork(None, [4] * 5, apply=False)
    assert want["status"][0] > 0 and want["count"] == 0
    p.fork([1, 1, 0, 4, -1], [4] * 5, apply=False, in_place=True)   # a row's end gives pages back
    assert p.fork([0, 1, 2, 3, 4], [4] * 5, apply=False, in_place=True)["status"][0] > 0
    assert all(np.array_equal(a, b) for a, b in zip(state, (p.table, p.lengths, p.refs)))
    for grow, most in (([1, 0, -1, 0, 0], 1), ([3, 0, 0, 0, 0], 2), ([25, 0, 0, 0, 0], 25)):
        want = p.fork(None, grow, most, apply=False)
        assert want["status"][1] > 0
    p.fork(None, [1, 0, 0, 0, 0])


def test_states_that_are_not_consistent():
    """Lengths and ids out of range: rows count as empty, ids are carried along
    and counted nowhere; nothing out of range is touched."""
    p = Pool(3, 6, 5, 8, empty=0)
    p.lengths[0], p.lengths[1] = -3, 5 * 8 + 1
    p.lengths[2] = 12
    p.table[2, 1] = p.pages + 5
    p.table[3, 0] = -2
    p.fork([0, 1, 2, 3, 2, 5], [0, 0, 1, 1, 2, 0], apply=False)
    p.compact()


@pytest.mark.parametrize("layout", ["tokens", "heads"])
@pytest.mark.parametrize("heads,dim,x", [(1, 8, "f16"), (3, 24, "bf16"), (8, 128, "bf16"), (5, 40, "e4m3"), (2, 16, "e4m3"),
                                         (4, 256, "f16")])
def test_layouts_and_types(layout, heads, dim, x):
    p = Pool(4, 6, 5, 20, heads=heads, dim=dim, x=x, layout=layout, layers=3)
    p.fork([0, 0, 0, 3, 3, 5], [1] * 6)
    p.compact()


def test_many_layers_and_none():
    p = Pool(5, 4, 4, 8, layers=128, heads=1, dim=8)
    p.fork([1, 1, 1, 1], [1] * 4)
    p.compact()
    q = Pool(6, 4, 4, 8, layers=0)
    q.fork([1, 1, 1, 1], [1] * 4)
    q.compact(in_place=True)


@pytest.mark.parametrize("rows,width,page,spare", [(1, 1, 1, 0), (4, 5, 4, 0), (9, 30, 2, 400), (64, 90, 1, 5000), (3, 4, 8, 9000),
                                                   (200, 100, 1, 40)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compactions(rows, width, page, spare, in_place):
    p = Pool(rows, rows, width, page, spare=spare, heads=1, dim=8)
    p.compact(in_place)
    p.compact(in_place)   # nothing left to move
    p.fork(p.rng.integers(-1, rows, rows), None)
    p.compact(in_place)


def test_copies():
    p = Pool(7, 3, 4, 16, spare=40)
    before = p.snapshot()
    pairs = [(0, 9, 16), (1, 10, 3), (2, 11, 0), (3, 12, 99), (4, 4, 16), (-1, 13, 4), (5, p.pages, 4), (6, 14, -2), (7, 15, 16)]
    t = p.dev(np.array(pairs))[0]
    p.lib.sgemv_pages_copy(p.caches, t, p.dev(np.array([8]))[0])
    p.check_copies(before, [(0, 9, 16), (1, 10, 3), (3, 12, 16)])
    p.lib.sgemv_pages_copy(p.caches, t)
    p.check_copies(before, [(0, 9, 16), (1, 10, 3), (3, 12, 16), (7, 15, 16)])
    p.lib.sgemv_pages_copy(p.caches, t, p.dev(np.array([-4]))[0])
    p.lib.sgemv_pages_copy(p.caches, t, p.dev(np.array([1 << 30]))[0])
    p.lib.sgemv_pages_copy(p.caches, t[:0])


def test_graph():
    """A captured fork in place goes on from the state it finds."""
    p = Pool(8, 8, 40, 4, spare=200)
    t, n, r = p.dev(p.table, p.lengths, p.refs)
    parents, grow = p.dev(np.arange(8), np.ones(8))
    e = lambda *s: torch.full(s, 99, dtype=torch.int32, device=DEV)  # noqa: E731
    slots, pairs, count, status = e(8, 1), e(8, 3), e(1), e(2)
    run = lambda: p.lib.sgemv_pages_fork(t, n, r, t, n, r, p.workspace, page_size=4, parents=parents, grow=grow,  # noqa: E731
                                         slots=slots, pairs=pairs, count=count, status=status, caches=p.caches)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for step in range(6):
        new = p.rng.integers(0, 8, 8)
        parents.copy_(torch.from_numpy(new.astype(np.int32)))
        want = oracle.pages_fork(t.cpu().numpy(), n.cpu().numpy(), r.cpu().numpy(), 4, new, [1] * 8, 1)
        before = p.snapshot()
        if step % 2:
            run()
        else:
            graph.replay()
        torch.cuda.synchronize()
        for name, x in {"table": t, "lengths": n, "refs": r, "slots": slots, "pairs": pairs}.items():
            assert np.array_equal(x.cpu().numpy(), want[name]), (step, name)
        p.check_copies(before, want["pairs"][:want["count"]].tolist())


@pytest.mark.parametrize("rows,width,page,spare", [(1025, 4, 3, None), (5, 6, 4, 7000), (40, 1700, 1, None), (8192, 3, 2, None)])
@pytest.mark.parametrize("in_place", [False, True])
def test_forks_past_one_workgroup(rows, width, page, spare, in_place):
    """More rows, pages or table entries than one workgroup plans in its LDS."""
    p = Pool(rows, rows, width, page, spare=spare, heads=1, dim=8, layers=1)
    for step in range(3):
        p.fork(p.rng.integers(-1, rows, rows) if step != 1 else None, p.rng.integers(0, 3, rows) if step else None, in_place=in_place)
    p.fork([rows - 1] * rows, [1] * rows, in_place=in_place)   # all from one, where it fits


def test_tables_and_slots_with_strides():
    """A table whose rows lie apart, in place, with the places behind its rows kept."""
    p = Pool(9, 5, 6, 8)
    wide = torch.full((5, 11), 5, dtype=torch.int32, device=DEV)
    wide[:, :6] = torch.from_numpy(p.table).to(DEV)
    _, n, r, par, grow = p.dev(p.table, p.lengths, p.refs, [4, 3, 2, 1, 1], [2, 1, 0, 1, 1])
    e = lambda *s: torch.full(s, 99, dtype=torch.int32, device=DEV)  # noqa: E731
    slots, pairs, count, status = e(5, 2), e(5, 3), e(1), e(2)
    want = oracle.pages_fork(p.table, p.lengths, p.refs, 8, [4, 3, 2, 1, 1], [2, 1, 0, 1, 1], 2)
    t = wide[:, :6]
    p.lib.sgemv_pages_fork(t, n, r, t, n, r, p.workspace, page_size=8, parents=par, grow=grow, slots=slots, pairs=pairs,
                           count=count, status=status, caches=p.caches)
    for name, x in {"table": t, "lengths": n, "refs": r, "slots": slots, "pairs": pairs}.items():
        assert np.array_equal(x.cpu().numpy(), want[name]), name
    assert (wide[:, 6:] == 5).all()
