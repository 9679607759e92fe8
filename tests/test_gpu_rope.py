"""Norms of the heads with the position rotation on the GPU, into rows and into the paged cache, against plain implementations
in 64 bits."""
import math

import pytest
import torch

import test_gpu_cache_fp4 as fp4
import test_gpu_decode as dec
from test_gpu_decode import BF, DEV, gen, moe, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def freqs(rot, base=10000.0):
    return [base ** (-2 * i / max(rot, 1)) for i in range(rot // 2)]


def reference(x, w, eps, pos, freq, axis, pairs):
    """(y, bound) in 64 bits of x [T, heads, D]; pos int [n_axes, T].  The bound counts what 32 bits lose before the rounding:
    the norm 2^-21 of a column (rsqrt 2 units, three products, a sum of D squares), the rotation 2^-21 of the pair (the phase
    as an fp32 fraction of half a turn 2^-24 pi, sine and cosine 2 units each, two products and a sum)."""
    T, _, D = x.shape
    R = 2 * len(freq)
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    bound = y.abs() * 2.0 ** -21
    if R:
        a = torch.stack([pos[axis[i] if axis else 0].double().cpu() * freq[i] for i in range(R // 2)], 1).to(DEV)[:, None]
        c, s = torch.cos(a), torch.sin(a)
        i = torch.arange(R // 2, device=DEV)
        i, j = (i, i + R // 2) if pairs == "half" else (2 * i, 2 * i + 1)
        out, b2 = y.clone(), bound.clone()
        out[..., i], out[..., j] = y[..., i] * c - y[..., j] * s, y[..., i] * s + y[..., j] * c
        b2[..., i] = b2[..., j] = (y[..., i].abs() + y[..., j].abs()) * 2.0 ** -20
        y, bound = out, b2
    return y, bound


def assert_rows(got, ref):
    y, bound = ref
    err = (got.double() - y).abs()
    tol = 2.0 ** -8 * y.abs() + 1.01 * bound + 1e-38
    assert torch.all(err <= tol), f"{float((err - tol).max()):.3e} above its bound"


SHAPES = [  # T, heads of q, of k, D, rotated columns, axes, pairs
    (1, 32, 8, 128, 128, 1, "half"),
    (1, 1, 1, 64, 64, 1, "adjacent"),
    (7, 4, 2, 128, 64, 1, "half"),
    (33, 7, 1, 64, 2, 1, "half"),
    (5, 3, 3, 128, 126, 1, "half"),
    (6, 8, 1, 64, 50, 2, "adjacent"),
    (300, 16, 4, 128, 128, 3, "half"),
    (4, 40, 5, 64, 0, 1, "half"),
    (65, 64, 64, 64, 36, 3, "half"),
]


@pytest.mark.parametrize("T,hq,hk,D,rot,axes,pairs", SHAPES)
@pytest.mark.parametrize("norm,w32", [(True, False), (True, True), (False, False)])
def test_rows(moe, T, hq, hk, D, rot, axes, pairs, norm, w32):  # noqa: F811
    g = gen(T * 1000 + D + rot)
    wide = (randn(g, T, (hq + 2 * hk + 1) * D) * torch.exp(randn(g, (hq + 2 * hk + 1) * D))).to(BF)
    q, k = wide[:, :hq * D].unflatten(1, (hq, D)), wide[:, (hq + 1) * D:(hq + 1 + hk) * D].unflatten(1, (hk, D))
    qw, kw = ((1 + 0.3 * randn(g, D)).to(torch.float32 if w32 else BF) if norm else None for _ in "qk")
    axis = [i % axes for i in range(rot // 2)] if axes > 1 else None
    pos = torch.randint(-50, 200000, (axes if rot // 2 >= axes else 1, T), generator=g, device=DEV).to(torch.int32)
    plan = moe.RotaryPlan(freqs(rot), axis, pairs, DEV)
    before = wide.clone()
    qo, ko = moe.moe_head_norm_rope(q, k, plan, pos, qw, kw, 1e-5)
    assert torch.equal(wide, before)
    for x, w, got in ((q, qw, qo), (k, kw, ko)):
        assert_rows(got, reference(x, w, 1e-5, pos, freqs(rot), axis, pairs))
    only_k = moe.moe_head_norm_rope(None, k, plan, pos, qw, kw, 1e-5)
    assert only_k[0] is None and torch.equal(only_k[1], ko)
    assert torch.equal(moe.moe_head_norm_rope(q, None, plan, pos, qw, kw, 1e-5)[0], qo)
    moe.moe_head_norm_rope(q, k, plan, pos, qw, kw, 1e-5, q_out=q, k_out=k)  # in place, in the wide rows
    assert torch.equal(q, qo) and torch.equal(k, ko)
    rest = torch.ones(wide.shape[1], dtype=torch.bool, device=DEV)
    rest[:hq * D] = rest[(hq + 1) * D:(hq + 1 + hk) * D] = False
    assert torch.equal(wide[:, rest], before[:, rest])


@pytest.mark.parametrize("pos", [0, 1, -1, 2 ** 17 - 1, 10 ** 6 + 1, 2 ** 31 - 1, -2 ** 31])
def test_far_positions_lose_nothing(moe, pos):  # noqa: F811
    """Against phases in rational arithmetic: a 64-bit angle at 2^31 keeps 22 bits behind the point, enough for the bound."""
    from fractions import Fraction
    D, freq = 64, [1.0, 0.77, 1e-3, 6.0, -0.4] + [10.0 ** -i for i in range(27)]
    two_pi = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
    x = torch.randn(1, 2, D, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    plan = moe.RotaryPlan(freq, device=DEV)
    got = moe.moe_head_norm_rope(x, None, plan, torch.tensor([pos], dtype=torch.int32, device=DEV))[0]
    a = torch.tensor([float(Fraction(f) * pos / two_pi % 1) * 2 * math.pi for f in freq], dtype=torch.float64, device=DEV)
    x0, x1 = x.double().chunk(2, -1)
    y = torch.cat([x0 * a.cos() - x1 * a.sin(), x0 * a.sin() + x1 * a.cos()], -1)
    bound = torch.cat([x0.abs() + x1.abs()] * 2, -1) * 2.0 ** -20
    assert_rows(got, (y, bound))


def test_zero_rows_nan_and_empty_calls(moe):  # noqa: F811
    D = 128
    x = torch.zeros(3, 2, D, dtype=BF, device=DEV)
    x[1, 1, 5], x[2, 0, 0] = float("nan"), float("inf")
    w = torch.ones(D, device=DEV)
    plan = moe.RotaryPlan(freqs(D), device=DEV)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    y = moe.moe_head_norm_rope(x, None, plan, pos, w)[0]
    assert torch.all(y[0] == 0) and torch.isnan(y[1, 1]).all() and torch.all(y[1, 0] == 0) and torch.all(y[2, 1] == 0)
    assert torch.isnan(y[2, 0, 0])
    for rows in (torch.empty(0, 2, D, dtype=BF, device=DEV), torch.empty(0, 5, 2, D, dtype=BF, device=DEV)):
        out = moe.moe_head_norm_rope(rows, rows, plan, pos[:0], w, w)
        assert out[0].shape == rows.shape


# ---------------------------------------------------------------------------------------------- into the cache
def make(moe, fmt, *args, **kw):  # noqa: F811
    return fp4.make_cache(moe, *args, **kw) if fmt == "mxfp4" else dec.make_cache(moe, *args[:4], fmt, **kw)


def stored(fmt, cache, b, n, which):
    return (fp4.rows_of if fmt == "mxfp4" else dec.rows_of)(cache, b, n, which)


def at_scale(fmt, u):
    """The value nearest to u (in a block's units) that the format holds."""
    if fmt == "mxfp8":
        step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(u / step) * step).clamp(-448, 448)
    step = torch.where(u.abs() < 2, 0.5, torch.where(u.abs() < 4, 1.0, 2.0).double())
    return (torch.round(u / step) * step).clamp(-6, 6)


def assert_stored(fmt, cache, b, n, which, ref, heads_from=None):
    """Rows n - len(ref) .. of request b hold ref: nearest values between those of ref's two ends, in scales of its maximum."""
    y, bound = ref
    m = y.shape[0]
    got = stored(fmt, cache, b, n, which)[n - m:]
    if fmt == "bf16":
        assert_rows(got, ref)
        return
    emax = 8 if fmt == "mxfp8" else 2
    blocks = y.abs().unflatten(-1, (-1, 32))
    d = 1.01 * bound.unflatten(-1, (-1, 32)) + 1e-45
    e = [(torch.frexp((blocks + z * d).clamp(min=0).amax(-1))[1] - 1 - emax).clamp(-127, 127) for z in (-1, 1)]
    at = fp4.at_of(cache, b, n)
    scale = getattr(cache, which + "_scales")[at][n - m:].int() - 127
    assert torch.all((scale >= e[0]) & (scale <= e[1]))
    unit = torch.exp2(scale.double()).repeat_interleave(32, -1)
    lo, hi = (at_scale(fmt, (y + z * d.flatten(-2)) / unit) * unit for z in (-1, 1))
    assert torch.all((got >= lo) & (got <= hi))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("lens,L,kv,group,D,page,rot,pairs", [
    ([9], 1, 1, 1, 64, 4, 64, "half"), ([3, 40, 0, 129, 4], 4, 2, 4, 128, 32, 128, "half"),
    ([300, 7], 7, 3, 2, 64, 48, 30, "adjacent"), ([70], 70, 8, 1, 128, 3, 64, "half")])
@pytest.mark.parametrize("given", [False, True])
def test_append_rotated(moe, fmt, lens, L, kv, group, D, page, rot, pairs, given):  # noqa: F811
    B, hq = len(lens), kv * group
    cache, g = make(moe, fmt, lens, kv, D, page, seed=sum(lens) + L)
    names = ("k", "v") + (("k_scales", "v_scales") if fmt != "bf16" else ())
    before = {n: getattr(cache, n).clone() for n in names}
    qkv = randn(g, B * L, (hq + 2 * kv) * D).to(BF).view(B, L, hq + 2 * kv, D)
    q, k, v = qkv.split((hq, kv, kv), dim=2)
    qw, kw = ((1 + 0.3 * randn(g, D)).to(BF) for _ in "qk")
    plan = moe.RotaryPlan(freqs(rot), None, pairs, DEV)
    pos = (cache.seq_lens[:, None] - L + torch.arange(L, device=DEV)).to(torch.int32)
    k_out = torch.empty(B, L, kv, D, dtype=BF, device=DEV)
    if given:
        pos = torch.randint(0, 10 ** 6, (B, L), generator=g, device=DEV).to(torch.int32)
    q_out = cache.append_rotated(q, k, v, plan, pos if given else None, qw, kw, 1e-6, k_out=k_out)
    cache.check()
    flat = pos.reshape(1, -1)
    ref_q = reference(q.reshape(B * L, hq, D), qw, 1e-6, flat, freqs(rot), None, pairs)
    ref_k = reference(k.reshape(B * L, kv, D), kw, 1e-6, flat, freqs(rot), None, pairs)
    assert_rows(q_out.view(B * L, hq, D), ref_q)
    assert_rows(k_out.view(B * L, kv, D), ref_k)
    touched = torch.zeros(cache.k.shape[:2], dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        m = min(n, L)
        if not m:
            continue
        rows = slice(b * L + L - m, b * L + L)
        assert_stored(fmt, cache, b, n, "k", tuple(t[rows] for t in ref_k))
        at = fp4.at_of(cache, b, n)
        touched[at[0][n - m:], at[1][n - m:]] = True
    for n, old in before.items():  # nothing else is written
        assert torch.equal(getattr(cache, n)[~touched].view(torch.uint8), old[~touched].view(torch.uint8))
    # the values are append's, and without norm and rotation so are the keys
    other = make(moe, fmt, lens, kv, D, page, seed=sum(lens) + L)[0]
    other.append(k, v)
    for n in names[1::2]:
        assert torch.equal(getattr(cache, n)[touched], getattr(other, n)[touched])
    still = moe.RotaryPlan([], None, pairs, DEV)
    assert cache.append_rotated(None, k, v, still) is None
    for n in names:
        assert torch.equal(getattr(cache, n)[touched], getattr(other, n)[touched])


def test_append_rotated_reports_bad_pages_and_lengths(moe):  # noqa: F811
    cache, g = make(moe, "mxfp4", [5, 9], 1, 64, 4, seed=8)
    k = randn(g, 2, 2, 1, 64).to(BF)
    plan = moe.RotaryPlan(freqs(64), device=DEV)
    cache.block_table[1, 2] = cache.k.shape[0]
    cache.append_rotated(k, k, k, plan)
    with pytest.raises(moe.MoEError, match="page index"):
        cache.check()
    cache.block_table[:] = 0
    cache.seq_lens[0] = cache.block_table.shape[1] * 4 + 1
    cache.append_rotated(k, k, k, plan)
    with pytest.raises(moe.MoEError, match="sequence length"):
        cache.check()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
def test_blocks_that_are_not_finite(moe, fmt):  # noqa: F811
    """A NaN or an infinity among the keys or values: MXFP4 keeps it as a block of NaN, the other formats as append does."""
    D, n = 64, 6
    cache = make(moe, fmt, [n], 1, D, 4)[0]
    other = make(moe, fmt, [n], 1, D, 4)[0]
    k = torch.ones(1, n, 1, D, dtype=BF, device=DEV)
    k[0, 1, 0, 3], k[0, 2, 0, 40], k[0, 3, 0, 5] = float("nan"), float("inf"), -float("inf")
    cache.append_rotated(None, k, k, moe.RotaryPlan([], device=DEV))
    other.append(k, k)
    at = fp4.at_of(cache, 0, n)
    for name in ("k", "v") + (("k_scales", "v_scales") if fmt != "bf16" else ()):
        assert torch.equal(getattr(cache, name)[at].view(torch.uint8), getattr(other, name)[at].view(torch.uint8))
    if fmt == "mxfp4":
        got = stored(fmt, cache, 0, n, "k")[:, 0]
        assert torch.isnan(got[1, :32]).all() and torch.isnan(got[2, 32:]).all() and torch.isnan(got[3, :32]).all()
        assert torch.equal(torch.isnan(got).sum(-1).cpu(), torch.tensor([0, 32, 32, 32, 0, 0]))


def test_on_another_stream_and_in_a_graph(moe):  # noqa: F811
    B, L, kv, D = 3, 2, 2, 128
    cache, g = make(moe, "mxfp4", [20, 3, 50], kv, D, 16, seed=4)
    qkv = randn(g, B, L, 8, D).to(BF)
    q, k, v = qkv.split((4, 2, 2), dim=2)
    plan = moe.RotaryPlan(freqs(D), device=DEV)
    w = torch.ones(D, device=DEV)
    want = cache.append_rotated(q, k, v, plan, None, w, w).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(cache.append_rotated(q, k, v, plan, None, w, w, stream=side), want) or side.synchronize()
    out = torch.empty_like(want)
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            cache.append_rotated(q, k, v, plan, None, w, w, q_out=out)
        cache.seq_lens.add_(5)  # the replay reads the lengths of its time
        graph.replay()
    side.synchronize()
    pos = (cache.seq_lens[:, None] - L + torch.arange(L, device=DEV)).reshape(1, -1)
    assert_rows(out.view(B * L, 4, D), reference(q.reshape(B * L, 4, D), w, 1e-6, pos, freqs(D), None, "half"))
