"""The pool of cache pages on the GPU against the rules carried out one request and one page at a time, and the copies of
page contents."""
import random

import pytest
import torch

from test_gpu_decode import BF, DEV, gen, moe, randn  # noqa: F401

pytestmark = pytest.mark.gpu

EMPTY, BAD_REQUEST = 4, 8


class Model:
    """The tables on the host, and the calls' rules as sentences."""

    def __init__(self, n_seqs, max_pages, n_pages, page):
        self.table = [[-1] * max_pages for _ in range(n_seqs)]
        self.lens, self.refs, self.page, self.max_pages = [0] * n_seqs, [0] * n_pages, page, max_pages
        self.status = 0

    def pages(self, n):
        return -(-n // self.page)

    def resize(self, new):
        cap = self.max_pages * self.page
        self.status |= any(not 0 <= n <= cap for n in new)
        new = [n if 0 <= n <= cap else old for n, old in zip(new, self.lens)]
        for b, n in enumerate(new):
            for j in range(self.pages(n), self.pages(self.lens[b])):
                self.refs[self.table[b][j]] -= 1
                self.table[b][j] = -1
        free = [p for p, r in enumerate(self.refs) if r == 0]
        copies, wanted, given = [(-1, -1)] * len(new), 0, []
        for b, n in enumerate(new):
            old = self.lens[b]
            if n <= old:
                continue
            copy = old % self.page != 0 and self.refs[self.table[b][old // self.page]] > 1
            want = self.pages(n) - self.pages(old) + copy
            take, wanted = free[wanted:wanted + want], wanted + want
            if want and wanted > len(free):
                self.status |= EMPTY
                new[b] = old
                continue
            given.append((b, copy, take))
        for b, copy, take in given:
            j = self.pages(self.lens[b]) - copy
            if copy:
                copies[b] = (self.table[b][j], take[0])
                self.refs[self.table[b][j]] -= 1
            for p in take:
                self.table[b][j], self.refs[p], j = p, 1, j + 1
        self.lens = new
        return copies

    def fork(self, src, dst):
        before, seen = list(self.lens), set()
        for a, b in zip(src, dst):
            ok = 0 <= a < len(before) and 0 <= b < len(before)
            if not ok or b in seen or before[b]:
                self.status |= BAD_REQUEST
                if ok:
                    seen.add(b)
                continue
            seen.add(b)
            n = self.pages(before[a])
            self.table[b][:n] = self.table[a][:n]
            for p in self.table[a][:n]:
                self.refs[p] += 1
            self.lens[b] = before[a]

    def compact(self, capacity):
        live, free = [p for p, r in enumerate(self.refs) if r], [p for p, r in enumerate(self.refs) if not r]
        moves = [(a, b) for a, b in zip(reversed(live), free) if a > b][:capacity]
        to = dict(moves)
        for b, n in enumerate(self.lens):
            for j in range(self.pages(n)):
                self.table[b][j] = to.get(self.table[b][j], self.table[b][j])
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        return moves + [(-1, -1)] * (capacity - len(moves))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def same(pool, model):
    assert pool.block_table.tolist() == model.table
    assert pool.seq_lens.tolist() == model.lens and pool.page_refs.tolist() == model.refs
    held = [0] * len(model.refs)
    for b, n in enumerate(model.lens):
        for j in range(model.pages(n)):
            held[model.table[b][j]] += 1
    assert held == model.refs
    assert int(pool.status.item()) == model.status
    pool.status.zero_()
    model.status = 0


@pytest.mark.parametrize("n_seqs,max_pages,n_pages,page", [(1, 1, 1, 1), (5, 7, 20, 4), (40, 9, 160, 16), (600, 5, 1500, 3),
                                                           (33, 300, 5003, 64), (8192, 2, 9001, 2)])
def test_random_histories(moe, n_seqs, max_pages, n_pages, page):  # noqa: F811
    """Growth, truncation, branches and compaction in random order, over pools that run out."""
    rng = random.Random(n_seqs)
    model, pool = Model(n_seqs, max_pages, n_pages, page), moe.PagePool.allocate(n_seqs, max_pages, n_pages, page, DEV)
    cap = max_pages * page
    for step in range(14 if n_seqs < 1000 else 6):
        what = rng.choice(["grow", "grow", "any", "fork", "compact", "free"])
        if what == "fork":
            n = rng.randint(0, n_seqs)
            src, dst = [rng.randint(-1, n_seqs) for _ in range(n)], [rng.randint(0, n_seqs) for _ in range(n)]
            model.fork(src, dst)
            pool.fork(i32(src), i32(dst))
        elif what == "compact":
            cap_moves = rng.choice([0, 1, 3, n_pages])
            want = model.compact(cap_moves)
            got = pool.compact(torch.full((cap_moves, 2), 77, dtype=torch.int32, device=DEV))
            assert [tuple(x) for x in got.tolist()] == want
        else:
            new = {"grow": lambda n: min(cap, n + rng.choice([0, 1, 2, page, 3 * page])),
                   "any": lambda n: rng.choice([0, n, rng.randint(0, cap), rng.randint(-2, cap + 2)]),
                   "free": lambda n: rng.choice([0, 0, n, n // 2])}[what]
            new = [new(n) for n in model.lens]
            want = model.resize(list(new))
            assert [tuple(x) for x in pool.resize(i32(new)).tolist()] == want
        same(pool, model)


def test_every_holder_of_a_page_takes_its_own(moe):  # noqa: F811
    model, pool = Model(4, 3, 12, 8), moe.PagePool.allocate(4, 3, 12, 8, DEV)
    for m, new in ((model, [12, 0, 0, 0]),):
        m.resize(new)
    pool.resize(i32([12, 0, 0, 0]))
    model.fork([0, 0, 0], [1, 2, 3])
    pool.fork(i32([0, 0, 0]), i32([1, 2, 3]))
    same(pool, model)
    assert [tuple(x) for x in pool.resize(i32([13, 14, 15, 12])).tolist()] == model.resize([13, 14, 15, 12])
    same(pool, model)
    assert pool.free_pages() == sum(r == 0 for r in model.refs)


def test_a_pool_that_runs_out_keeps_the_requests_length(moe):  # noqa: F811
    pool = moe.PagePool.allocate(3, 4, 4, 2, DEV)
    pool.resize(i32([2, 8, 2]))
    assert pool.seq_lens.tolist() == [2, 0, 0]  # two and three wait: the pages that the second wanted are not passed on
    with pytest.raises(moe.MoEError, match="more pages than are free"):
        pool.check()
    pool.resize(i32([2, 4, 0]))
    pool.check()
    assert pool.block_table[1, :2].tolist() == [1, 2]


def test_bad_tables_are_reported_and_left_alone(moe):  # noqa: F811
    pool = moe.PagePool.allocate(2, 4, 8, 2, DEV)
    pool.resize(i32([5, 4]))
    pool.block_table[0, 1] = 8
    pool.block_table[1, 0] = -5
    refs = pool.page_refs.clone()
    pool.resize(i32([0, 4]))
    with pytest.raises(moe.MoEError, match="page index"):
        pool.check()
    assert int((refs - pool.page_refs).sum()) == 2
    pool.seq_lens[1] = 9
    pool.compact(torch.empty(8, 2, dtype=torch.int32, device=DEV))
    with pytest.raises(moe.MoEError, match="sequence length"):
        pool.check()


def test_empty_calls(moe):  # noqa: F811
    pool = moe.PagePool.allocate(0, 3, 0, 16, DEV)
    assert pool.resize(i32([])).shape == (0, 2)
    pool.fork(i32([]), i32([]))
    pool.compact(torch.empty(0, 2, dtype=torch.int32, device=DEV))
    pool = moe.PagePool.allocate(3, 0, 0, 16, DEV)
    pool.resize(i32([0, 0, 0]))
    pool.compact(torch.empty(4, 2, dtype=torch.int32, device=DEV))
    pool.check()
    moe.moe_copy_pages([], torch.empty(4, 2, dtype=torch.int32, device=DEV))


# ---------------------------------------------------------------------------------------------- contents
def layer(moe, fmt, n_pages, page, kv, D, layout="rows", seed=0):  # noqa: F811
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    g = gen(seed)
    inner = {"rows": (n_pages, page, kv), "heads": (n_pages, kv, page), "heads first": (kv, n_pages, page),
             "wide": (n_pages, page, kv + 1)}[layout]

    def tensor(cols, dtype):
        t = torch.randint(0, 256, (*inner, cols * (2 if dtype is BF else 1)), generator=g, device=DEV, dtype=torch.uint8)
        t = t.view(dtype)
        return {"rows": t, "heads": t.transpose(1, 2), "heads first": t.permute(1, 2, 0, 3), "wide": t[:, :, :kv]}[layout], t

    cols = {"bf16": D, "mxfp8": D, "mxfp4": D // 2}[fmt]
    kinds = [(cols, BF if fmt == "bf16" else torch.uint8)] * 2 + ([(D // 32, torch.uint8)] * 2 if fmt != "bf16" else [])
    views, whole = zip(*[tensor(*x) for x in kinds])
    return moe.PagedKVCache(views[0], views[1], table, lens, *views[2:]), whole


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("layout", ["rows", "heads", "heads first", "wide"])
@pytest.mark.parametrize("page,kv,D", [(1, 1, 64), (16, 3, 64), (5, 2, 128), (64, 8, 128)])
def test_copy_pages(moe, fmt, layout, page, kv, D):  # noqa: F811
    n_pages = 23
    caches, wholes = zip(*[layer(moe, fmt, n_pages, page, kv, D, layout, seed=i) for i in range(3)])
    pairs = [(-1, -1), (3, 0), (22, 1), (-1, 5), (3, 2), (7, 21)]
    want = []
    for c, whole in zip(caches, wholes):
        copy = [w.clone() for w in whole]
        for x in zip(("k", "v", "k_scales", "v_scales"), copy):
            view = getattr(c, x[0])
            as_view = x[1].view(torch.uint8).as_strided(
                (*view.shape[:3], view.shape[3] * view.element_size()), (*[s * view.element_size() for s in view.stride()[:3]], 1))
            for a, b in pairs:
                if a >= 0:
                    as_view[b] = as_view[a]
        want.append(copy)
    moe.moe_copy_pages(caches, i32(pairs))
    for c, whole, copy in zip(caches, wholes, want):
        c.check()
        for a, b in zip(whole, copy):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_copy_many_pages_of_many_layers(moe):  # noqa: F811
    """More tensors than one launch takes, and more pairs than one window, of mixed formats."""
    n_pages = 1400
    layers = [layer(moe, ("bf16", "mxfp8", "mxfp4")[i % 3], n_pages, 4, 2, 64, seed=i) for i in range(40)]
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(0))
    pairs = order.view(-1, 2).to(torch.int32)
    pairs[::3] = -1
    before = [[w.clone() for w in whole] for _, whole in layers]
    moe.moe_copy_pages([c for c, _ in layers], pairs.to(DEV))
    a, b = (pairs[pairs[:, 0] >= 0, i].long().to(DEV) for i in (0, 1))
    for (_, whole), old in zip(layers, before):
        for x, y in zip(whole, old):
            y[b] = y[a]
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_copy_reports_pages_outside_a_cache(moe):  # noqa: F811
    cache, whole = layer(moe, "mxfp8", 5, 4, 2, 64)
    before = [w.clone() for w in whole]
    for bad in ([5, 0], [0, 5], [0, -1]):
        moe.moe_copy_pages([cache], i32([bad]))
        with pytest.raises(moe.MoEError, match="page index"):
            cache.check()
    assert all(torch.equal(a, b) for a, b in zip(whole, before))


def test_branches_attend_like_requests_of_their_own(moe):  # noqa: F811
    """A request, its branch with other tokens, truncation and compaction: attention reads what each should hold."""
    page, kv, D, n_pages = 16, 2, 64, 40
    pool = moe.PagePool.allocate(3, 8, n_pages, page, DEV)
    caches = [moe.PagedKVCache.allocate(n_pages, page, kv, D, pool.block_table, pool.seq_lens, f) for f in ("bf16", "mxfp4")]
    alone = [moe.PagedKVCache.allocate(24, page, kv, D, torch.arange(24, dtype=torch.int32, device=DEV).view(3, 8),
                                       torch.zeros(3, dtype=torch.int32, device=DEV), f) for f in ("bf16", "mxfp4")]
    g = gen(3)

    def step(new, L, k, v):
        copies = pool.resize(i32(new))
        moe.moe_copy_pages(caches, copies)
        for c in caches:
            c.append(k, v)
        for c in alone:
            c.seq_lens.copy_(i32(new))
            c.append(k, v)

    k, v = (randn(g, 3, 37, kv, D).to(BF) for _ in "kv")
    step([37, 0, 20], 37, k, v)
    pool.fork(i32([0]), i32([1]))
    for c in alone:  # the branch by hand
        for t in (c.k, c.v) + ((c.k_scales, c.v_scales) if c.k_scales is not None else ()):
            t[8:11] = t[0:3]
    k, v = (randn(g, 3, 3, kv, D).to(BF) for _ in "kv")
    step([40, 40, 23], 3, k, v)
    moves = pool.compact(torch.empty(n_pages // 2, 2, dtype=torch.int32, device=DEV))
    moe.moe_copy_pages(caches, moves)
    pool.resize(i32([38, 40, 0]))
    for c in alone:
        c.seq_lens.copy_(i32([38, 40, 0]))
    pool.check()
    assert int(pool.page_refs.max()) == 2 and pool.free_pages() == n_pages - 4
    q = randn(g, 3, 2, 4, D).to(BF)
    for c, a in zip(caches, alone):
        assert torch.equal(c.attend(q), a.attend(q))
        c.check()


def test_a_captured_step_takes_pages_at_every_replay(moe):  # noqa: F811
    pool = moe.PagePool.allocate(2, 30, 64, 4, DEV)
    cache = moe.PagedKVCache.allocate(64, 4, 1, 64, pool.block_table, pool.seq_lens, "mxfp4")
    new, copies = torch.zeros(2, dtype=torch.int32, device=DEV), torch.empty(2, 2, dtype=torch.int32, device=DEV)
    k = torch.ones(2, 3, 1, 64, dtype=BF, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            torch.add(pool.seq_lens, 3, out=new)
            pool.resize(new, copies)
            moe.moe_copy_pages([cache], copies)
            cache.append(k, k)
        for _ in range(9):
            graph.replay()
    side.synchronize()
    pool.check()
    cache.check()
    assert pool.seq_lens.tolist() == [27, 27] and pool.free_pages() == 64 - 14
    assert sorted(pool.block_table[:, :7].flatten().tolist()) == list(range(14))
