"""The decode-step operators at the edges of their contracts: workspaces that many calls share, rows that hold NaN,
scales at the ends of E8M0, prompts of many row tiles."""
import ctypes
import math
import os
import sys

import pytest
import torch

import oracle
import synth
from gpu_support import assert_close, bf16_to_f64, x_to_device
from test_gpu_decode import BF, DEV, HALF_ULP, attend_ref, check_attend, fill, gen, make_cache, moe, randn  # noqa: F401

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


# ---------------------------------------------------------------------------------------------- workspaces
def attend_c(moe, cache, q, ws):
    """moe_paged_attention through the C call, in a workspace of the caller's."""
    B, L, H, D = q.shape
    out, lse = torch.full_like(q, float("nan")), torch.full((B, L, H), float("nan"), device=DEV)
    a = moe.moe_attention_t(q.data_ptr(), out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), 0, 0, H, L, D ** -0.5)
    assert moe.lib().moe_paged_attention(cache._ref, ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    cache.check()
    return out, lse


def test_one_workspace_serves_calls_of_any_shape(moe):  # noqa: F811
    """Parts of one call must not lie where another one counts: requests, heads, row tiles and widths that differ."""
    shapes = [  # lens, kv, group, L, D, format
        ([20000], 8, 4, 1, 128, "bf16"),
        ([300 + 17 * i for i in range(64)], 8, 4, 8, 128, "mxfp8"),
        ([4000, 9000], 2, 16, 4, 64, "bf16"),
        ([700] * 40, 1, 16, 5, 64, "mxfp8"),
        ([20000], 8, 4, 1, 128, "bf16"),
        ([50] * 150, 1, 4, 1, 64, "bf16"),
        ([30000], 1, 8, 1, 128, "mxfp8"),
    ]
    calls, size = [], 0
    for i, (lens, kv, group, L, D, fmt) in enumerate(shapes):
        cache, g = make_cache(moe, lens, kv, D, 64, fmt, seed=200 + i)
        fill(cache, g, lens)
        q = (1.5 * randn(g, len(lens), L, kv * group, D)).to(BF)
        size = max(size, moe.lib().moe_paged_attention_workspace(cache._ref, kv * group, L))
        calls.append((cache, q))
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV)  # what is not a counter may hold anything
    ws[:moe.MOE_ATTENTION_COUNTER_BYTES] = 0
    for cache, q in calls + calls[::-1]:
        fresh = torch.zeros(size, dtype=torch.uint8, device=DEV)
        want, got = attend_c(moe, cache, q, fresh), attend_c(moe, cache, q, ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert not torch.isnan(got[0]).any() and not torch.isnan(got[1]).any()
        assert torch.all(ws[:moe.MOE_ATTENTION_COUNTER_BYTES] == 0)


def layer_of(moe, d, f, E, k, seed, max_T=8, **kw):  # noqa: F811
    """A layer of random weights (any codes; scales near 1 / sqrt(columns))."""
    g = gen(seed)

    def codes(n, rows, cols):
        e = 127 - 2 - cols.bit_length() // 2
        return (torch.randint(0, 256, (n, rows, cols // 2), dtype=torch.uint8, device=DEV, generator=g),
                torch.randint(e - 1, e + 1, (n, rows, cols // 32), dtype=torch.uint8, device=DEV, generator=g))

    ex, sh = (moe.DeviceExperts(*codes(n, 2 * f, d), *codes(n, d, f)) for n in (E, 1))
    return moe.MoELayer(d, f, E, k, ex, sh, randn(g, E, d) * d ** -0.5, 0.05 * randn(g, E), max_T=max_T, device=DEV, **kw)


def test_layers_of_other_shapes_may_share_a_workspace(moe):  # noqa: F811
    """What one layer leaves in the workspace is no counter of another's: one-kernel calls and ordinary ones in turn."""
    d = 512
    layers = [layer_of(moe, d, f, E, k, 300 + f) for f, E, k in ((256, 16, 4), (1024, 8, 2), (128, 64, 6))]
    xs = [randn(gen(310 + T), T, d).to(BF) for T in (1, 3, 8)]
    want = [[(ly.forward_few(x), ly.forward(x)) for x in xs] for ly in layers]
    shared = torch.full((max(moe.moe_workspace_size(ly.cfg, 8) for ly in layers),), 0xA5, dtype=torch.uint8, device=DEV)
    for ly in layers:
        moe.moe_set_workspace(ly.h, shared, 8)
    for _ in range(2):
        for i, x in enumerate(xs):
            for ly, w in zip(layers, want):
                assert torch.equal(ly.forward_few(x), w[i][0])
            for ly, w in zip(layers, want):
                assert torch.equal(ly.forward(x), w[i][1])
                assert torch.equal(ly.forward_few(x), w[i][0])
    for ly in layers:
        ly.check()


# ---------------------------------------------------------------------------------------------- rows that hold NaN
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("lens", [[90, 6], [30000, 500]])  # units of one block; units that many blocks share
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_lse_of_a_row_that_holds_nan_is_nan(moe, fmt, lens, bad):  # noqa: F811
    """-inf is for rows that see nothing: who joins parts by lse would drop such a row's NaN."""
    kv, group, L, D = 2, 4, 2, 64
    cache, g = make_cache(moe, lens, kv, D, 16, fmt, seed=400)
    fill(cache, g, lens)
    q = randn(g, 2, L, kv * group, D).to(BF)

    def attend():
        lse = torch.full(q.shape[:3], 7.0, device=DEV)
        return cache.attend(q, lse=lse), lse

    want, want_lse = attend()
    q[0, 1, 2, 5] = bad
    got, lse = attend()
    assert torch.isnan(got[0, 1, 2]).all() and torch.isnan(lse[0, 1, 2])
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[0, 1, 2] = True
    assert torch.equal(got[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    q[0, 1, 2, 5] = 0.5
    n = lens[1]  # every key of request 1 and head 0
    pos = torch.arange(n)
    at = (cache.tab[1, pos // 16].long().to(DEV), (pos % 16).to(DEV))
    cache.k[(*at, torch.zeros(n, dtype=torch.long, device=DEV))] = math.nan if fmt == "bf16" else 0x7F
    got, lse = attend()
    assert torch.isnan(got[1, :, :group]).all() and torch.isnan(lse[1, :, :group]).all()
    assert torch.isfinite(lse[1, :, group:]).all() and torch.isfinite(lse[0]).all()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("L", [1, 2, 3])
def test_a_nan_value_of_negligible_weight_reaches_the_rows_that_see_it(moe, fmt, L):  # noqa: F811
    """A row's own newest token, with a weight that fp32 cannot hold: its NaN counts as it does at every other place."""
    lens, D = [100, 41], 64
    cache, g = make_cache(moe, lens, 1, D, 16, fmt, seed=430)
    fill(cache, g, lens)
    q = (4 + randn(g, 2, L, 4, D).abs()).to(BF)
    for b, n in enumerate(lens):
        page, row = int(cache.tab[b, (n - 1) // 16]), (n - 1) % 16
        if fmt == "bf16":
            cache.k[page, row], cache.v[page, row, 0, 9] = -300, math.nan
        else:
            cache.k[page, row], cache.k_scales[page, row] = 0xFE, 127  # -448
            cache.v[page, row, 0, 9] = 0x7F
    out = cache.attend(q)
    assert torch.isnan(out[:, -1, :, 9]).all()
    out[:, -1, :, 9] = 0
    assert torch.isfinite(out).all()


# ---------------------------------------------------------------------------------------------- the ends of E8M0
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L", [1, 12])
def test_attend_keys_of_the_smallest_scale(moe, D, L):  # noqa: F811
    """Byte 0 is 2^-127, not 0: keys near 2^-125 against queries near 2^120."""
    lens = [100, 700]
    cache, g = make_cache(moe, lens, 1, D, 16, "mxfp8", seed=420)
    k = (randn(g, 2, 700, 1, D) * 2.0 ** -125).to(BF)
    v = randn(g, 2, 700, 1, D).to(BF)
    cache.append(k, v)
    assert int(cache.k_scales[cache.tab[0, 0], 0].max()) == 0
    q = (randn(g, 2, L, 4, D) * 2.0 ** 120).to(BF)
    out, _ = check_attend(cache, q, lens, scale=8.0)
    assert not torch.allclose(out[0, 0, 0].float(), out[0, 0, 1].float(), rtol=0.1, atol=0.1)  # the scores matter


@pytest.mark.parametrize("which", ["s13", "s2"])
def test_few_weights_of_the_smallest_scale(moe, which):  # noqa: F811
    """Byte 0 of the experts' scales is 2^-127, as moe_forward reads it: large x against W13, the layer's limit against
    W2."""
    wl = synth.WORKLOADS["tiny"].with_T(4)
    inp, ids, wts, _ = oracle.margin_filtered_layer(wl, 7)
    for e in (inp.experts, inp.shared):
        getattr(e, which)[...] = 0
    # h of order 1 to 100: x 2^117 against the scales 2^-127 of W13, x 2^4 against its own
    bits = (torch.from_numpy(inp.x.view("int16")).view(BF).float() * 2.0 ** (117 if which == "s13" else 4)).to(BF)
    inp.x = bits.view(torch.int16).numpy().view("uint16")
    ids, wts, margin = oracle.route(inp.x, inp.router_w, inp.router_bias, wl.k, wl.route_scale)
    assert (margin >= oracle.MARGIN_MIN).all()
    layer = moe.MoELayer.from_host(inp, device=DEV, max_T=4)
    x = x_to_device(inp.x)
    y_ref = oracle.layer(inp.x, ids, wts, inp.experts, inp.shared, wl.swiglu_limit)
    assert abs(y_ref).max() > 2.0 ** -118
    out = layer.forward_few(x)
    layer.check()
    assert_close(bf16_to_f64(layer.forward(x)), y_ref, f"{which} = 0, moe_forward")
    assert_close(bf16_to_f64(out), y_ref, f"{which} = 0")


# ---------------------------------------------------------------------------------------------- streams
def test_results_on_another_stream_do_not_take_the_current_streams_memory(moe):  # noqa: F811
    """A block just freed on the current stream may have work pending there: a call on another stream leaves it alone."""
    cache, g = make_cache(moe, [70, 500], 2, 128, 16, "bf16", seed=460)
    fill(cache, g, [70, 500])
    q = randn(g, 2, 2, 8, 128).to(BF)
    ly = layer_of(moe, 512, 256, 8, 2, 461)
    x = randn(g, 3, 512).to(BF)
    side = torch.cuda.Stream()
    for call in (lambda **kw: cache.attend(q, **kw), lambda **kw: ly.forward_few(x, **kw), lambda **kw: ly.forward(x, **kw)):
        want = call()
        freed = [torch.empty_like(want) for _ in range(8)]
        at = {t.data_ptr() for t in freed}
        del freed
        side.wait_stream(torch.cuda.current_stream())
        for stream in (side, side.cuda_stream):
            got = call(stream=stream)
            side.synchronize()
            assert got.data_ptr() not in at and torch.equal(got, want)


def test_graphs_and_eager_calls_of_one_cache_may_overlap(moe):  # noqa: F811
    """Captured calls count in workspaces of their own: two graphs captured on a stream, and eager calls there, all at
    once."""
    lens = [20000, 300, 9000]
    cache, g = make_cache(moe, lens, 2, 128, 64, "bf16", seed=470)
    fill(cache, g, lens)
    q = [randn(g, 3, 1, 8, 128).to(BF) for _ in range(3)]
    want = [cache.attend(t) for t in q]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], [torch.empty_like(t) for t in q]
    with torch.cuda.stream(side):
        cache.attend(q[0], outs[0])  # the stream's own workspace exists before the captures
        for i in (0, 1):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                cache.attend(q[i], outs[i])
            graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(20):
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            graphs[0].replay()
        graphs[1].replay()
        with torch.cuda.stream(side):
            cache.attend(q[2], outs[2])
        torch.cuda.synchronize()
        for t, w in zip(outs, want):
            assert torch.equal(t, w)
    cache.check()


def test_attend_in_a_workspace_of_the_callers(moe):  # noqa: F811
    lens = [20000, 300]
    cache, g = make_cache(moe, lens, 2, 128, 64, "mxfp8", seed=480)
    fill(cache, g, lens)
    q1, q4 = (randn(g, 2, L, 8, 128).to(BF) for L in (1, 4))
    want = [cache.attend(q) for q in (q1, q4)]
    ws = cache.attention_workspace(8, 4)
    for _ in range(2):
        for q, w in zip((q1, q4), want):
            assert torch.equal(cache.attend(q, workspace=ws), w)
    with pytest.raises(moe.MoEError) as err:
        cache.attend(randn(g, 2, 16, 8, 128).to(BF), workspace=ws)  # larger row tiles
    assert err.value.status == 3


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L,limit", [(4, 11e6), (8, 17e6), (16, 33e6)])  # row tiles of 16, 32 and 64
def test_a_workspace_holds_two_parts_a_block(moe, fmt, D, L, limit):  # noqa: F811
    """No more than the blocks of the form need, and nothing is written past it: long requests split over all blocks."""
    lens = [40000, 25000, 31000]
    cache, g = make_cache(moe, lens, 2, D, 64, fmt, seed=490)
    fill(cache, g, lens)
    q = randn(g, 3, L, 8, D).to(BF)
    n = moe.lib().moe_paged_attention_workspace(cache._ref, 8, L)
    assert 0 < n < limit * D / 128
    guarded = torch.full((n + (1 << 20),), 0xA5, dtype=torch.uint8, device=DEV)
    guarded[:moe.MOE_ATTENTION_COUNTER_BYTES] = 0
    out, _ = attend_c(moe, cache, q, guarded[:n])
    assert torch.equal(out, cache.attend(q)) and torch.all(guarded[n:] == 0xA5)


def test_the_example_waits_for_its_set_up(moe, monkeypatch, capsys):  # noqa: F811
    """Its steps run on a stream of their own; the lengths and inputs are written on the current one, here after a pause."""
    import decode_block
    blocks = []

    def built_late(*args, _build=decode_block.random_block, **kw):
        blocks.append(_build(*args, **kw))
        torch.cuda._sleep(200_000_000)  # 0.1 s of the current stream, in front of what main() still writes there
        return blocks[-1]

    monkeypatch.setattr(decode_block, "random_block", built_late)
    monkeypatch.setattr(sys, "argv", ["decode_block.py", "--requests", "2", "--tokens", "2", "--context", "100", "--steps", "4"])
    decode_block.main()
    torch.cuda.synchronize()
    assert blocks[0].cache.seq_lens.tolist() == [100 + 2 * (3 + 4)] * 2
    assert "us a step" in capsys.readouterr().out


def test_append_to_a_table_without_pages_reports_the_lengths(moe):  # noqa: F811
    """No page can hold the new tokens: the length is above the bound, as in any other table."""
    pages = torch.zeros(4, 16, 1, 64, dtype=BF, device=DEV)
    lens = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    cache = moe.PagedKVCache(pages, pages.clone(), torch.empty(2, 0, dtype=torch.int32, device=DEV), lens)
    new = torch.ones(2, 1, 1, 64, dtype=BF, device=DEV)
    cache.append(new, new)
    with pytest.raises(moe.MoEError, match="sequence length"):
        cache.check()
    assert torch.all(pages == 0)
    lens.zero_()
    cache.append(new, new)
    cache.check()


# ---------------------------------------------------------------------------------------------- the few-token layer's limits
@pytest.mark.parametrize("T,d", [(2, 39680), (4, 19200), (7, 10496), (8, 8960)])
def test_few_takes_rows_up_to_the_stated_width(moe, T, d):  # noqa: F811
    """include/moe_decode.h gives the widest d_model for every number of rows: that one runs, the next is refused."""
    ly = layer_of(moe, d, 128, 4, 2, 510 + T)
    x = randn(gen(520 + T), T, d).to(BF)
    want = ly.forward(x)
    got = ly.forward_few(x)
    ly.check()
    # the same arithmetic but for the fp16 rounding of moe_forward's rows and the order of fp32 sums
    assert_close(bf16_to_f64(got), bf16_to_f64(want), f"{T} rows of {d}")
    wider = layer_of(moe, d + 256, 128, 4, 2, 530 + T)
    with pytest.raises(moe.MoEError) as err:
        wider.forward_few(randn(gen(540 + T), T, d + 256).to(BF))
    assert err.value.status == 2


# ---------------------------------------------------------------------------------------------- prompts
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("lens,kv,group,L,D,page", [
    ([300, 777], 2, 4, 300, 128, 16),      # a prompt on an empty and on a filled cache: 19 row tiles of 64
    ([2000], 1, 4, 2000, 64, 48),          # 125 row tiles
    ([100, 0, 333, 64], 1, 16, 100, 64, 64),  # prompts shorter than the longest of them
    ([1023], 2, 1, 257, 128, 128),         # one row over
])
def test_attend_prompts(moe, fmt, lens, kv, group, L, D, page):  # noqa: F811
    cache, g = make_cache(moe, lens, kv, D, page, fmt, seed=450 + L)
    fill(cache, g, lens)
    q = (1.5 * randn(g, len(lens), L, kv * group, D)).to(BF)
    out, lse = check_attend(cache, q, lens)
    assert torch.equal(cache.attend(q), out)
    if L > 2:  # the last rows alone: the same attention in another form of the kernel, to the same bounds
        check_attend(cache, q[:, -2:].contiguous(), lens)


@pytest.mark.parametrize("B,L", [(1, 1), (2, 2), (3, 4)])  # 1 and 4 rows: forward_few; 12: forward
def test_the_blocks_moe_half_against_the_layer_in_64_bits(moe, B, L):  # noqa: F811
    """Every row: the rows that the block's second norm makes, with their own routing, through the oracle's layer."""
    import decode_block
    d, f, E, k = 512, 256, 8, 2
    block = decode_block.random_block(d, f, E, k, 8, 2, 64, B, 64, L, page=16, fmt="bf16", seed=11 * B)
    ly = block.layer
    host = [synth.ExpertWeights(*(getattr(e, n).cpu().numpy() for n in ("w13", "s13", "w2", "s2")))
            for e in (ly.experts, ly.shared_w)]
    g, seen = gen(500 + B), 0
    for _ in range(3):
        x, res = randn(g, B * L, d).to(BF), randn(g, B * L, d).to(BF)
        rows = []
        for name in ("forward", "forward_few"):  # what the block hands to its layer
            def spy(y, call=getattr(moe.MoELayer, name).__get__(ly)):
                rows.append(y.clone())
                return call(y)
            setattr(ly, name, spy)
        block.cache.seq_lens.add_(L)
        out, stream = block.step(x, res, L)
        ly.check()
        assert len(rows) == 1
        t = stream.double()
        y2 = t / torch.sqrt((t * t).mean(-1, keepdim=True) + block.eps) * block.norm_moe.double()
        # the norm is of the unrounded sum: its rounding to the stream (2^-9 a value) moves a row's rms by less, and y2 is
        # rounded once more
        assert torch.all((rows[0].double() - y2).abs() <= 2 * (HALF_ULP + 2.0 ** -17) * y2.abs() + 2.0 ** -9 * y2.abs())
        bits = rows[0].cpu().view(torch.int16).numpy().view("uint16")
        ids, wts, margin = oracle.route(bits, ly.router_w.cpu().numpy(), ly.router_bias.cpu().numpy(), k, 1.5)
        sure = margin >= oracle.MARGIN_MIN
        ref = oracle.layer(bits, ids, wts, *host, 10.0)
        seen += int(sure.sum())
        if sure.any():
            assert_close(bf16_to_f64(out)[sure], ref[sure], f"{B} x {L}")
    assert seen >= 2 * B * L  # of three steps' rows


@pytest.mark.parametrize("D", [64, 128])
def test_attend_values_of_the_smallest_scale_beside_a_hidden_nan(moe, D):  # noqa: F811
    """Values near 2^-123 in blocks of byte 0, with a NaN that the first rows do not see: taken one by one they are the same
    values."""
    cache, g = make_cache(moe, [50], 1, D, 16, "mxfp8", seed=560)
    k = randn(g, 1, 50, 1, D).to(BF)
    cache.append(k, (randn(g, 1, 50, 1, D).clamp(-3, 3) * 2.0 ** -123).to(BF))
    page = cache.tab[0].tolist()
    assert max(int(cache.v_scales[p].where(cache.v_scales[p] < 200, 0).max()) for p in page[:3]) == 0
    q = randn(g, 1, 3, 2, D).to(BF)
    want = cache.attend(q).float()[0, :2] * 2.0 ** 123
    assert want.abs().max() > 2.0 ** -3
    cache.v[page[49 // 16], 49 % 16] = 0x7F  # the last row's own token
    got = cache.attend(q).float()[0, :2] * 2.0 ** 123
    # two forms of the same products, each rounded to bf16 (below 2^-126 to a fixed step of 2^-133)
    assert torch.all((got - want).abs() <= 2 * HALF_ULP * want.abs() + 2.0 ** -9)


# ---------------------------------------------------------------------------------------------- far rows
def test_norm_rows_beyond_32_bit_offsets(moe):  # noqa: F811
    """2.5 G elements; and the most rows that a call takes."""
    T, d = 600_011, 4096
    g = gen(570)
    base = randn(g, 4096, d).to(BF)
    x = torch.empty(T, d, dtype=BF, device=DEV)
    for i in range(0, T, 4096):
        x[i:i + 4096] = base[:min(4096, T - i)]
    w = (1 + 0.1 * randn(g, d)).to(BF)
    y, yq = torch.empty_like(x), torch.empty(T, d, dtype=torch.uint8, device=DEV)
    ys = torch.empty(T, d // 32, dtype=torch.uint8, device=DEV)
    moe.moe_add_rms_norm(x, None, w, 1e-6, None, y, yq, ys)
    n = T % 4096
    for t in (y.view(torch.int16), yq, ys):
        assert torch.equal(t[-n:], t[:n]) and torch.equal(t[4096 * 100:4096 * 101], t[:4096])
    del x, y, yq, ys
    T = 2 ** 31 - 1
    x = torch.ones(T, 8, dtype=BF, device=DEV)
    x[-1] = 2
    moe.moe_add_rms_norm(x, None, torch.ones(8, device=DEV), 0.0, None, x)
    assert torch.all(x[:: 2 ** 16] == 1) and torch.all(x[-9:] == 1)  # every row has one value: the norm is 1
