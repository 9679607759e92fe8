"""Argument checks of the 4-bit cache, the head norms with rotation and the page pool: every refusal is made on the host,
before any work, without a GPU."""
import ctypes

import pytest
import torch

P = 4096  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def m():
    import __graft_entry__ as g
    g.build_cuda()
    import block_scaled_fp4_sqrt_gb300 as mod
    return mod


def fill(s, values):
    for k, v in values.items():
        setattr(s, k, v)
    return s


def cache(m, **kw):
    return fill(m.moe_kv_cache_t(), {**dict(
        k=P, v=P, k_s=P, v_s=P, block_table=P, seq_lens=P, status=P, page_stride=2048, row_stride=128, head_stride=128,
        format=4, n_pages=4, page_size=16, n_kv_heads=1, head_dim=128, n_seqs=2, max_pages=2), **kw})


@pytest.mark.parametrize("kw", [dict(format=3), dict(format=5), dict(head_dim=96), dict(row_stride=16), dict(page_stride=-32),
                                dict(k=P + 8), dict(v=P + 1), dict(k_s=None), dict(v_s=None), dict(k_s=P + 2), dict(k=None),
                                dict(head_stride=32), dict(seq_lens=None), dict(max_pages=1 << 30)])
def test_four_bit_caches_are_refused_by_every_call(m, kw):
    L, c = m.lib(), cache(m, **kw)
    att = m.moe_attention_t(P, P, None, P, 1 << 30, 0, 0, 4, 1, 1.0)
    assert L.moe_kv_append(ctypes.byref(c), P, 0, P, 0, 1, None) in (1, 2)
    assert L.moe_last_error()
    assert L.moe_paged_attention(ctypes.byref(c), ctypes.byref(att), None) in (1, 2)
    assert L.moe_paged_attention_workspace(ctypes.byref(c), 4, 1) == 0
    assert L.moe_head_norm_rope(ctypes.byref(c), ctypes.byref(rope(m, head_dim=kw.get("head_dim", 128))), None) in (1, 2)
    at = (ctypes.POINTER(m.moe_kv_cache_t) * 1)(ctypes.pointer(c))
    assert L.moe_copy_pages(at, 1, P, 1, None) in (1, 2)


def test_four_bit_caches_that_span_too_much(m):
    c = cache(m, page_stride=1 << 40)
    att = m.moe_attention_t(P, P, None, P, 1 << 30, 0, 0, 4, 1, 1.0)
    assert m.lib().moe_paged_attention(ctypes.byref(c), ctypes.byref(att), None) == 2


# ---------------------------------------------------------------------------------------------- head norms, rotation
def rope(m, **kw):
    return fill(m.moe_head_rope_t(), {**dict(
        q=P, k=P, v=P, q_out=2 * P, k_out=3 * P, q_weight=P, k_weight=P, turns=P, axis=None, positions=P, T=2, L=1, n_q_heads=4,
        n_kv_heads=1, head_dim=128, rot_dim=128, pairs=0, n_axes=1, weight_f32=0, eps=1e-6), **kw})


ROPE_BAD = [dict(head_dim=96), dict(head_dim=256), dict(rot_dim=-2), dict(rot_dim=130), dict(rot_dim=63), dict(pairs=2),
            dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(n_axes=0), dict(n_axes=257), dict(n_q_heads=-1),
            dict(n_q_heads=70000), dict(q=P + 2), dict(k=P + 8), dict(q_out=P + 4), dict(k_out=P + 1), dict(q_stride=100),
            dict(q_stride=516), dict(k_stride=64), dict(q_weight=P + 8), dict(k_weight=P + 2), dict(turns=P + 4),
            dict(positions=P + 2), dict(q=None), dict(q_out=None), dict(turns=None)]


@pytest.mark.parametrize("kw", ROPE_BAD)
@pytest.mark.parametrize("with_cache", [False, True])
def test_rope_refuses(m, kw, with_cache):
    c = cache(m) if with_cache else None
    ref = ctypes.byref(c) if with_cache else None
    assert m.lib().moe_head_norm_rope(ref, ctypes.byref(rope(m, **kw)), None) in (1, 2), kw
    assert b"moe_head_norm_rope" in m.lib().moe_last_error()


def test_rope_refuses_what_its_form_lacks(m):
    L, c = m.lib(), cache(m)
    for kw in (dict(T=-1), dict(k_out=None), dict(k=None), dict(positions=None), dict(n_axes=2, position_stride=1),
               dict(q=None, q_out=None, k=None, k_out=None)):
        assert L.moe_head_norm_rope(None, ctypes.byref(rope(m, **kw)), None) == 1, kw
    for kw in (dict(L=-1), dict(k=None), dict(v=None), dict(n_kv_heads=2), dict(head_dim=64), dict(v=P + 2), dict(v_stride=8)):
        assert L.moe_head_norm_rope(ctypes.byref(c), ctypes.byref(rope(m, **kw)), None) == 1, kw
    assert L.moe_head_norm_rope(None, None, None) == 1
    assert L.moe_head_norm_rope(None, ctypes.byref(rope(m, T=0)), None) == 0  # nothing to do
    assert L.moe_head_norm_rope(ctypes.byref(c), ctypes.byref(rope(m, L=0)), None) == 0
    assert L.moe_head_norm_rope(None, ctypes.byref(rope(m, T=0x7FFFFFFF)), None) == 2
    assert L.moe_head_norm_rope(None, ctypes.byref(rope(m, n_q_heads=40000, n_kv_heads=20000)), None) == 2


# ---------------------------------------------------------------------------------------------- pages
def pool(m, **kw):
    return fill(m.moe_page_pool_t(), {**dict(block_table=P, seq_lens=P, page_refs=P, status=P, n_seqs=4, max_pages=8,
                                             n_pages=32, page_size=16), **kw})


@pytest.mark.parametrize("kw", [dict(n_seqs=-1), dict(max_pages=-1), dict(n_pages=-1), dict(page_size=0), dict(block_table=None),
                                dict(seq_lens=None), dict(page_refs=None), dict(block_table=P + 1), dict(seq_lens=P + 2),
                                dict(page_refs=P + 3), dict(status=P + 1), dict(n_seqs=8193), dict(max_pages=1 << 28),
                                dict(n_pages=(1 << 30) + 1)])
def test_pools_are_refused_by_every_call(m, kw):
    L, p = m.lib(), pool(m, **kw)
    assert L.moe_pages_fork(ctypes.byref(p), P, P, 1, None) in (1, 2)
    assert L.moe_pages_resize(ctypes.byref(p), P, P, None) in (1, 2)
    assert L.moe_pages_compact(ctypes.byref(p), P, 4, None) in (1, 2)


def test_page_calls_refuse(m):
    L, p = m.lib(), pool(m)
    for args in ((None, P, 1), (P, None, 1), (P, P, -1), (P, P, 5), (P + 2, P, 1), (P, P + 1, 1)):
        assert L.moe_pages_fork(ctypes.byref(p), *args, None) == 1, args
    for args in ((None, P), (P, None), (P + 2, P), (P, P + 4)):
        assert L.moe_pages_resize(ctypes.byref(p), *args, None) == 1, args
    for args in ((None, 4), (P, -1), (P + 4, 4)):
        assert L.moe_pages_compact(ctypes.byref(p), *args, None) == 1, args
    at = (ctypes.POINTER(m.moe_kv_cache_t) * 1)(ctypes.pointer(cache(m)))
    for args in ((None, 1, P, 1), (at, -1, P, 1), (at, 1, None, 1), (at, 1, P, -1), (at, 1, P + 4, 1)):
        assert L.moe_copy_pages(*args, None) == 1, args
    assert L.moe_pages_fork(None, P, P, 1, None) == L.moe_pages_resize(None, P, P, None) == 1
    assert L.moe_copy_pages(at, 1, None, 0, None) == L.moe_copy_pages(None, 0, P, 3, None) == 0  # nothing to do


# ---------------------------------------------------------------------------------------------- the binding, traced
from test_decode_binding import OnGpu, cache as cache_of, expand, m as traced, zeros  # noqa: E402,F401

BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture
def b(traced, monkeypatch):  # noqa: F811
    return traced


def plan(b, rot=64, axes=None, index=0):
    p = b.RotaryPlan([0.5 ** i for i in range(rot // 2)], axes, device="cpu")
    p.turns = OnGpu(p.turns, index)
    return p


def test_the_formats_of_a_cache_follow_from_its_tensors(b, monkeypatch):
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, _r=torch.zeros, **k: _r(*a, **k))
    table, lens = zeros(2, 2, dtype=I32), zeros(2, dtype=I32)

    def make(cols, dtype, scale_cols, **kw):
        k, s = zeros(4, 16, 3, cols, dtype=dtype), zeros(4, 16, 3, scale_cols, dtype=U8) if scale_cols else None
        return b.PagedKVCache(k, k, table, lens, s, s, **kw)

    for (cols, dtype, sc), want in (((128, BF, 0), (0, 128)), ((64, U8, 2), (1, 64)), ((128, U8, 4), (1, 128)),
                                    ((64, U8, 4), (4, 128)), ((32, U8, 2), (4, 64))):
        c = make(cols, dtype, sc)
        assert (c.format, c.head_dim) == want
        assert (c._c.head_stride, c._c.row_stride, c._c.page_stride) == (want[1], 3 * want[1], 48 * want[1])
    for bad in ((64, U8, 3), (64, U8, 8), (64, BF, 4), (16, U8, 2)):
        with pytest.raises(ValueError):
            make(*bad)
    wide = OnGpu(torch.zeros(4, 16, 3, 160, dtype=U8)[..., :64])  # rows of the scales do not lie alike
    with pytest.raises(ValueError, match="strides"):
        b.PagedKVCache(wide, wide, table, lens, *[zeros(4, 16, 3, 4, dtype=U8)] * 2)


def test_rotary_plans(b):
    import math
    p = b.RotaryPlan([1.0, -0.25, 2 * math.pi], device="cpu")
    t = [x % 2 ** 64 for x in p.turns.tolist()]
    # 2^64 / (2 pi) = 2935890503282001226.496.., a quarter of it 733972625820500306.624..
    assert t[0] == 2935890503282001226 and t[1] == 2 ** 64 - 733972625820500307
    assert min(t[2], 2 ** 64 - t[2]) < 2 ** 12  # a whole turn but for what 2 pi loses in 64 bits
    assert (p.rot_dim, p.n_axes) == (6, 1)
    assert b.RotaryPlan([1, 2, 3], [0, 2, 1], device="cpu").n_axes == 3
    for bad in (dict(inv_freq=[float("nan")]), dict(inv_freq=[float("inf")]), dict(inv_freq=[1.0], pairs="both"),
                dict(inv_freq=[1.0], axis_of=[0, 1]), dict(inv_freq=[1.0], axis_of=[-1]), dict(inv_freq=[1.0], axis_of=[256])):
        with pytest.raises(ValueError):
            b.RotaryPlan(device="cpu", **bad)


def test_head_norm_rope_passes_strides_and_refuses_the_rest(b):
    wide = OnGpu(torch.zeros(6, 10 * 64, dtype=BF))
    view = lambda lo, h: OnGpu(wide.t[:, lo * 64:(lo + h) * 64].unflatten(1, (h, 64)))  # noqa: E731
    q, k, pos, w = view(0, 4), view(6, 2), zeros(1, 6, dtype=I32), zeros(64)
    good = dict(q=q, k=k, rope=plan(b), positions=pos, q_weight=w, k_weight=w, q_out=zeros(6, 4, 64), k_out=zeros(6, 2, 64))
    b.moe_head_norm_rope(**good)
    a = b.library.calls[-1][1][1]._obj if hasattr(b.library.calls[-1][1][1], "_obj") else b.library.calls[-1][1][1]
    assert (a.T, a.n_q_heads, a.n_kv_heads, a.head_dim, a.rot_dim) == (6, 4, 2, 64, 64)
    assert (a.q_stride, a.k_stride, a.q_out_stride, a.k_out_stride, a.weight_f32) == (640, 640, 256, 128, 0)
    b.moe_head_norm_rope(**{**good, "k": None, "k_out": None})
    b.moe_head_norm_rope(**{**good, "q": OnGpu(zeros(2, 3, 4, 64).t), "q_out": zeros(2, 3, 4, 64)})  # rows in two dimensions
    calls = len(b.library.calls)
    other = zeros(6, 4, 64, index=1)
    for kw in (dict(q=None), dict(q=expand(zeros(1, 4, 64), 6, 4, 64)), dict(q=zeros(5, 4, 64)), dict(q=zeros(6, 4, 128)),
               dict(q=zeros(6, 4, 64, dtype=torch.float32)), dict(q=other), dict(q_out=zeros(6, 2, 64)),
               dict(q_out=expand(zeros(1, 4, 64), 6, 4, 64)), dict(q=OnGpu(torch.zeros(6, 64, 4, dtype=BF).transpose(1, 2))),
               dict(q=OnGpu(torch.zeros(6, 8, 64, dtype=BF)[:, ::2])), dict(positions=None), dict(positions=zeros(1, 5, dtype=I32)),
               dict(positions=zeros(1, 6, dtype=torch.int64)), dict(positions=OnGpu(torch.zeros(6, 2, dtype=I32).t()[:1])),
               dict(q_weight=zeros(32)), dict(q_weight=zeros(64, dtype=torch.float32)), dict(k_weight=zeros(64, dtype=torch.float16)),
               dict(rope=plan(b, axes=[i % 3 for i in range(32)])), dict(rope=plan(b, index=1)), dict(q=None, k=None),
               dict(q=OnGpu(torch.zeros(3, 2, 4, 64, dtype=BF).transpose(0, 1)), q_out=zeros(2, 3, 4, 64))):
        with pytest.raises(ValueError):
            b.moe_head_norm_rope(**{**good, **kw})
    assert len(b.library.calls) == calls


def test_append_rotated_passes_strides_and_refuses_the_rest(b):
    c = cache_of(b, n_seqs=3, heads=2, head_dim=64)
    qkv = torch.zeros(3, 2, 8, 64, dtype=BF)
    q, k, v = (OnGpu(t) for t in qkv.split((4, 2, 2), dim=2))
    good = dict(q=q, k_new=k, v_new=v, rope=plan(b), q_weight=zeros(64), k_weight=zeros(64), q_out=zeros(3, 2, 4, 64))
    assert c.append_rotated(**good) is good["q_out"]
    a = b.library.calls[-1][1][1]
    assert (a.L, a.q_stride, a.k_stride, a.v_stride, a.q_out_stride, a.positions, a.k_out) == (2, 512, 512, 512, 256, None, None)
    assert c.append_rotated(None, k, v, plan(b)) is None
    calls = len(b.library.calls)
    for kw in (dict(q=zeros(3, 1, 4, 64)), dict(v_new=zeros(3, 1, 2, 64)), dict(k_new=zeros(3, 2, 1, 64)), dict(q=None),
               dict(q_out=zeros(3, 2, 2, 64)), dict(k_out=zeros(3, 1, 2, 64)), dict(k_new=expand(zeros(1, 1, 2, 64), 3, 2, 2, 64)),
               dict(positions=zeros(1, 5, dtype=I32)), dict(q_weight=zeros(128)), dict(q=zeros(3, 2, 4, 64, index=1)),
               dict(rope=plan(b, index=1))):
        with pytest.raises(ValueError):
            c.append_rotated(**{**good, **kw})
    assert len(b.library.calls) == calls


def test_pools_pass_what_fits_and_refuse_the_rest(b, monkeypatch):
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, _r=torch.zeros, **k: _r(*a, **k))
    table, lens, refs = zeros(3, 4, dtype=I32), zeros(3, dtype=I32), zeros(20, dtype=I32)
    p = b.PagePool(table, lens, refs, 16)
    new, copies = zeros(3, dtype=I32), zeros(3, 2, dtype=I32)
    assert p.resize(new, copies) is copies and p.compact(zeros(7, 2, dtype=I32)).shape == (7, 2)
    p.fork(zeros(2, dtype=I32), zeros(2, dtype=I32))
    assert [c[0] for c in b.library.calls] == ["moe_pages_resize", "moe_pages_compact", "moe_pages_fork"]
    calls = len(b.library.calls)
    for bad in (lambda: p.resize(zeros(2, dtype=I32), copies), lambda: p.resize(zeros(3, dtype=torch.int64), copies),
                lambda: p.resize(new, zeros(2, 2, dtype=I32)), lambda: p.resize(OnGpu(torch.zeros(6, dtype=I32)[::2]), copies),
                lambda: p.resize(zeros(3, dtype=I32, index=1), copies), lambda: p.compact(zeros(7, dtype=I32)),
                lambda: p.compact(OnGpu(torch.zeros(2, 7, dtype=I32).t())), lambda: p.fork(zeros(2, dtype=I32), zeros(3, dtype=I32)),
                lambda: p.fork(zeros(2, 1, dtype=I32), zeros(2, 1, dtype=I32)), lambda: b.PagePool(table, zeros(2, dtype=I32), refs, 16),
                lambda: b.PagePool(zeros(3, 4), lens, refs, 16), lambda: b.PagePool(OnGpu(torch.zeros(4, 3, dtype=I32).t()), lens, refs, 16),
                lambda: b.PagePool(table, lens, zeros(20, dtype=I32, index=1), 16),
                lambda: b.PagePool(zeros(8193, 1, dtype=I32), zeros(8193, dtype=I32), refs, 16),
                lambda: b.moe_copy_pages([], zeros(3, dtype=I32)), lambda: b.moe_copy_pages([], zeros(3, 2, dtype=torch.int64)),
                lambda: b.moe_copy_pages([], OnGpu(torch.zeros(2, 3, dtype=I32).t())), lambda: b.moe_copy_pages([], zeros(3, 2, dtype=I32, index=1))):
        with pytest.raises((ValueError, IndexError)):
            bad()
    c = cache_of(b)
    c._index, c._at = 1, None
    with pytest.raises(ValueError, match="cache lies"):
        b.moe_copy_pages([c], zeros(3, 2, dtype=I32))
    assert len(b.library.calls) == calls
