"""Calls of the cache's operators at the ends of what they allow: pages far into a large pool, several streams and graphs at
once, the same index and the same tensor twice."""
import pytest
import torch

import test_gpu_cache_fp4 as fp4
from test_gpu_decode import BF, DEV, gen, moe, randn  # noqa: F401
from test_gpu_pages import i32
from test_gpu_rope import freqs

pytestmark = pytest.mark.gpu


def cache_at(moe, n_pages, pages, n, page, kv, D):  # noqa: F811
    return moe.PagedKVCache.allocate(n_pages, page, kv, D, i32([pages]), i32([n]), "mxfp4")


def test_pages_far_into_a_pool(moe):  # noqa: F811
    """Codes beyond 2^32 bytes: writer, rotation, attention and copies do what they do in the first pages, bit for bit."""
    n, page, kv, D = 1500, 64, 8, 128
    need = -(-n // page)
    n_pages = 2 ** 32 // (page * kv * D // 2) + 2 * need
    last = list(range(n_pages - 1, n_pages - 1 - need, -1))
    near, far = cache_at(moe, 2 * need, list(range(need)), n, page, kv, D), cache_at(moe, n_pages, last, n, page, kv, D)
    g = gen(3)
    q, k, v = (randn(g, 1, n, h, D).to(BF) for h in (2 * kv, kv, kv))
    w = (1 + 0.3 * randn(g, D)).to(BF)
    plan = moe.RotaryPlan(freqs(D), device=DEV)
    outs = []
    for c in (near, far):
        turned = c.append_rotated(q, k, v, plan, None, w, w)
        outs.append((turned, c.attend(turned), c.attend(turned[:, -1:])))
        c.append(k[:, -2:], v[:, -2:])
        outs[-1] += (c.attend(turned[:, -3:]),)
        c.check()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    names = ("k", "v", "k_scales", "v_scales")
    for t in names:
        assert torch.equal(getattr(near, t)[:need], getattr(far, t)[last])
        assert not getattr(far, t)[:need].any()
    moe.moe_copy_pages([far], i32([(p, j) for j, p in enumerate(last)]))
    for t in names:
        assert torch.equal(getattr(near, t)[:need], getattr(far, t)[:need])
    moe.moe_copy_pages([far], i32([(j, p - need) for j, p in enumerate(last)]))
    far.block_table.sub_(need)
    assert torch.equal(far.attend(turned[:, -3:]), outs[1][3])
    far.check()


def test_axes_that_a_call_does_not_have_count_as_its_last(moe):  # noqa: F811
    T, D, rot = 19, 64, 48
    x = randn(gen(5), T, 3, D).to(BF)
    plan = moe.RotaryPlan(freqs(rot), [0, 1, 2] * 8, device=DEV)
    pos = torch.randint(-100, 10 ** 6, (3, T), generator=gen(6), device=DEV).to(torch.int32)
    want = moe.moe_head_norm_rope(x, None, plan, pos)[0]
    plan.axis[2::6] = 3
    plan.axis[5::6] = 255
    assert torch.equal(moe.moe_head_norm_rope(x, None, plan, pos)[0], want)


def test_attention_on_two_streams_and_in_two_graphs_at_once(moe):  # noqa: F811
    """Lengths that are split over many blocks, so that every call joins parts in its workspace."""
    calls = []
    for i, (lens, kv, group, L, D) in enumerate([([9000, 700], 2, 4, 1, 128), ([5000, 20, 6000], 4, 8, 5, 64)]):
        cache, g = fp4.make_cache(moe, lens, kv, D, 32, seed=i)
        fp4.fill(cache, g, lens)
        calls.append((cache, randn(g, len(lens), L, kv * group, D).to(BF)))
    want = [c.attend(q) for c, q in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(20):
        for (c, q), s, to in zip(calls, streams, got):
            with torch.cuda.stream(s):
                to.append(c.attend(q))
    torch.cuda.synchronize()
    assert all(torch.equal(t, w) for to, w in zip(got, want) for t in to)

    outs, graphs = [torch.empty_like(w) for w in want], []
    for (c, q), s, out in zip(calls, streams, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            for _ in range(10):
                c.attend(q, out)
    for _ in range(3):
        for out in outs:
            out.fill_(7)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip(outs, want))
    for c, _ in calls:
        c.check()


def test_the_same_request_and_tensor_twice(moe):  # noqa: F811
    pool = moe.PagePool.allocate(6, 4, 20, 8, DEV)
    pool.resize(i32([20, 0, 0, 0, 3, 0]))
    assert pool.page_refs.tolist() == [1] * 4 + [0] * 16
    pool.fork(i32([0, 0, 0]), i32([1, 2, 3]))  # three branches of one request
    pool.check()
    assert pool.page_refs[:4].tolist() == [4, 4, 4, 1] and pool.seq_lens.tolist() == [20, 20, 20, 20, 3, 0]
    for src, dst in (([0, 4], [5, 5]), ([5], [5])):  # two pairs with one branch: the first; a branch of itself: length 0, nothing
        pool.fork(i32(src), i32(dst))
        if len(src) == 2:
            with pytest.raises(moe.MoEError, match="fork"):
                pool.check()
            assert pool.seq_lens[5] == 20 and pool.page_refs[:4].tolist() == [5, 5, 5, 1]
            pool.resize(i32([20, 20, 20, 20, 3, 0]))
        pool.check()
    state = [t.clone() for t in (pool.block_table, pool.seq_lens, pool.page_refs)]
    assert torch.all(pool.resize(pool.seq_lens) == -1)  # the lengths that there are: nothing changes
    pool.check()
    assert all(torch.equal(a, b) for a, b in zip(state, (pool.block_table, pool.seq_lens, pool.page_refs)))

    cache = moe.PagedKVCache.allocate(20, 8, 2, 64, pool.block_table, pool.seq_lens)
    cache.k.normal_(), cache.v.normal_()
    want_k, want_v = cache.k.clone(), cache.v.clone()
    want_k[[7, 9]], want_v[[7, 9]] = want_k[[2, 2]], want_v[[2, 2]]
    moe.moe_copy_pages([cache, cache], i32([(2, 7), (-1, -1), (2, 9)]))  # one source twice, one cache twice
    cache.check()
    assert torch.equal(cache.k, want_k) and torch.equal(cache.v, want_v)


@pytest.mark.parametrize("group,L", [(11, 3), (4, 10), (16, 3), (7, 7), (8, 8), (13, 5), (3, 65)])
def test_attention_of_many_rows_a_head(moe, group, L):  # noqa: F811
    """33 to 195 rows a key-value head: what a row tile of any size has to get right."""
    lens, kv, D = [5000, 70, 0, 130], 2, 64
    cache, g = fp4.make_cache(moe, lens, kv, D, 48, seed=group)
    fp4.fill(cache, g, lens)
    fp4.check_attend(cache, (1.5 * randn(g, len(lens), L, kv * group, D)).to(BF), lens)
    for lo, hi in ((99, 135), (98, 127), (0, 3)):
        fp4.test_attend_values_of_any_scale(moe, D, group, L, lo, hi)
    for order in ("growing", "falling"):
        fp4.test_attend_large_scores_move_the_maximum(moe, D, group, L, order)


@pytest.mark.parametrize("L", [10, 16, 31])
def test_nan_blocks_and_many_rows(moe, L):  # noqa: F811
    fp4.test_attend_nan_blocks_reach_only_the_rows_that_see_them(moe, 64, L)


@pytest.mark.parametrize("D,group,L", [(64, 4, 1), (128, 4, 1), (128, 4, 8), (64, 4, 8)])
def test_blocks_of_zeros_among_the_values(moe, D, group, L):  # noqa: F811
    """Zeros of either sign under any scale byte but 255 add nothing; tiny and large blocks of the same tokens still do."""
    lens, kv = [400, 33], 2
    cache, g = fp4.make_cache(moe, lens, kv, D, 16, seed=D + L)
    fp4.fill(cache, g, lens)
    for b, n in enumerate(lens):
        at = fp4.at_of(cache, b, n)
        codes, scales = cache.v[at].unflatten(-1, (-1, 16)), cache.v_scales[at]
        kind = torch.randint(0, 5, scales.shape, generator=g, device=DEV)
        kind[n // 2:][kind[n // 2:] > 2] = 1  # half of the tokens hold nothing but zeros and ordinary blocks
        for i, (code, scale) in {1: (0x00, 0), 2: (0x80, 254), 3: (None, 60), 4: (None, 150)}.items():
            scales[kind == i] = scale
            if code is not None:
                codes[kind == i] = code
        cache.v[at], cache.v_scales[at] = codes.flatten(-2), scales
    q = randn(g, 2, L, kv * group, D).to(BF)
    want, _ = fp4.check_attend(cache, q, lens)
    at = fp4.at_of(cache, 0, lens[0])
    cache.v_scales[at[0][-1], at[1][-1], 0, 0], cache.v[at[0][-1], at[1][-1], 0, :16] = 255, 0  # the newest token of one head
    out = cache.attend(q)
    hit = torch.zeros_like(q, dtype=torch.bool)
    hit[0, -1, :group, :32] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[0, :-1], want[0, :-1]) and torch.equal(out[1], want[1])
