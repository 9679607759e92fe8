"""The paged cache held in 4 bits (MXFP4) on the GPU, its writer and its attention, against plain implementations in 64
bits."""
import math

import pytest
import torch

from test_gpu_decode import BF, DEV, gen, moe, randn  # noqa: F401

pytestmark = pytest.mark.gpu

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def quantize_ref(x):
    """(packed codes, scale bytes) of x [..., n] in 64 bits: exponent floor(log2 amax) - 2 in [-127, 127], byte 0 for a zero
    block, 255 (and codes 0) for one with a NaN or an infinity; nearest code, ties to even, saturating."""
    b = x.double().cpu().unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 3).clamp(-127, 127), torch.full(amax.shape, -127, dtype=torch.int32))
    u = (b * torch.exp2(-e.double())[..., None]).flatten(-2)
    mag = E2M1[:8]
    d = (u.abs()[..., None] - mag).abs()
    near = d == d.amin(-1, keepdim=True)  # one code, or two at a tie: the even one
    code = torch.where(near[..., 0::2].any(-1), near[..., 0::2].int().argmax(-1) * 2, near.int().argmax(-1))
    odd_nearer = near.int().sum(-1) == 1
    code = torch.where(odd_nearer, near.int().argmax(-1), code)
    code = (code | (torch.signbit(u).int() << 3)).to(torch.uint8)
    scale = torch.where(bad, 255, e + 127).to(torch.uint8)
    code = torch.where(bad.repeat_interleave(32, -1), torch.zeros_like(code), code)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(DEV), scale.to(DEV)


def make_cache(moe, lens, kv, D, page, seed=0, layout="rows", spare=2):  # noqa: F811
    """A cache of random contents whose unused rows are NaN; pages of the requests in random order."""
    g = gen(seed)
    per = [-(-n // page) for n in lens]
    n_pages = sum(per) + spare
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.full((len(lens), max(per + [1]) + 1), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
    inner = (n_pages, kv, page) if layout == "heads" else (n_pages, page, kv)
    fix = (lambda t: t.transpose(1, 2)) if layout == "heads" else (lambda t: t)
    k, v = (fix(torch.full((*inner, D // 2), 0x77, dtype=torch.uint8, device=DEV)) for _ in "kv")
    ks, vs = (fix(torch.full((*inner, D // 32), 255, dtype=torch.uint8, device=DEV)) for _ in "kv")
    cache = moe.PagedKVCache(k, v, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), ks, vs)
    cache.tab = table
    return cache, g


def at_of(cache, b, n):
    pos = torch.arange(n)
    page = cache.k.shape[1]
    return cache.tab[b, pos // page].long().to(DEV), (pos % page).to(DEV)


def rows_of(cache, b, n, which):
    """Request b's first n rows as fp64 [n, kv, D]."""
    at = at_of(cache, b, n)
    c, s = getattr(cache, which)[at], getattr(cache, which + "_scales")[at]
    v = E2M1.to(DEV)[torch.stack([c & 15, c >> 4], -1).flatten(-2).long()]
    scale = torch.where(s == 255, torch.full((), float("nan"), dtype=torch.float64, device=DEV), torch.exp2(s.double() - 127))
    return v * scale.repeat_interleave(32, -1)


def fill(cache, g, lens, k_gain=1.0, v_gain=1.0):
    """Append the whole context of every request at once."""
    L = max(lens)
    if L == 0:
        return None, None
    k = (k_gain * randn(g, len(lens), L, cache.n_kv_heads, cache.head_dim)).to(BF)
    v = (v_gain * randn(g, len(lens), L, cache.n_kv_heads, cache.head_dim)).to(BF)
    cache.append(k, v)
    return k, v


def reference(cache, q, lens, scale):
    """out, lse in 64 bits, and the error bounds that go with them.

    Scores: q in fp16 with its row's power of two errs by 2^-17 of the row's maximum at most, the products are exact, their
    fp32 sums of D terms err by D 2^-24 of the magnitudes.  p and z carry that relative error and 2^-20 for the exponential and
    the sums; p is rounded to fp16, by 2^-11 of itself or 2^-31 of the row's largest weight; the output once to bf16, 2^-8."""
    B, L, H, D = q.shape
    kv = cache.n_kv_heads
    out = torch.zeros(B, L, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, L, H), -math.inf, dtype=torch.float64, device=DEV)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        K, V = (rows_of(cache, b, n, x).transpose(0, 1) for x in "kv")  # [kv, n, D]
        qq = q[b].double().unflatten(1, (kv, H // kv)).permute(1, 0, 2, 3)  # [kv, L, g, D]
        seen = (torch.arange(n, device=DEV) < (n - L + 1 + torch.arange(L, device=DEV))[:, None])[None, :, None]
        s = torch.einsum("hlgd,htd->hlgt", qq, K) * scale
        err = D * 2.0 ** -24 * torch.einsum("hlgd,htd->hlgt", qq.abs(), K.abs())
        err = err + 2.0 ** -17 * qq.abs().amax(-1)[..., None] * K.abs().sum(-1)[:, None, None]
        err = (abs(scale) * err).masked_fill(~seen, 0.0).amax(-1) + 2.0 ** -20
        s = s.masked_fill(~seen, -math.inf)
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - z.clamp(min=-1e300)[..., None])
        o, a = torch.einsum("hlgt,htd->hlgd", p, V), torch.einsum("hlgt,htd->hlgd", p, V.abs())
        floor = torch.einsum("hlgt,htd->hlgd", seen.expand_as(p).double() * p.amax(-1, keepdim=True), V.abs()) * 2.0 ** -31
        t = 2.0 ** -8 * 1.01 * o.abs() + (2.0 ** -11 + 2 * err[..., None]) * 1.01 * a + floor + 1e-37
        place = lambda x: x.permute(1, 0, 2, *range(3, x.dim())).flatten(1, 2)  # noqa: E731
        out[b], lse[b], tol[b] = place(o), place(z), place(t)
        tol_lse[b] = place(err + 2.0 ** -21 * z.abs())
    return out, lse, tol, tol_lse


def check_attend(cache, q, lens, scale=None, **kw):
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    out = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
    assert cache.attend(q, out, lse, scale, **kw) is out
    torch.cuda.synchronize()
    cache.check()
    ref, rl, tol, tl = reference(cache, q, lens, q.shape[-1] ** -0.5 if scale is None else scale)
    err = (out.double() - ref).abs()
    assert torch.all(err <= tol), f"out: {float((err - tol).max()):.3e} above its bound"
    dead = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), dead) and torch.all(out[dead] == 0)
    el = (lse.double() - rl).abs()[~dead]
    assert torch.all(el <= tl[~dead]), f"lse: {float((el - tl[~dead]).max()):.3e} above its bound"
    return out, lse


# ---------------------------------------------------------------------------------------------- writer
@pytest.mark.parametrize("layout", ["rows", "heads"])
@pytest.mark.parametrize("lens,kv,D,page", [([1], 1, 64, 1), ([0, 5, 64, 65], 2, 128, 16), ([7, 300, 2], 3, 64, 48),
                                            ([129], 8, 128, 3)])
def test_append_writes_every_token_exactly(moe, lens, kv, D, page, layout):  # noqa: F811
    cache, g = make_cache(moe, lens, kv, D, page, seed=sum(lens), layout=layout)
    before = {n: getattr(cache, n).clone() for n in ("k", "v", "k_scales", "v_scales")}
    L = max(lens)
    wide = randn(g, len(lens) * L, 5 * kv * D).to(BF)  # views of a fused projection
    wide[::3, ::5] *= 100
    wide[1::7] = 0
    k, v = (wide[:, i * kv * D:(i + 1) * kv * D].unflatten(0, (len(lens), L)).unflatten(-1, (kv, D)) for i in (1, 3))
    cache.append(k, v)
    cache.check()
    touched = torch.zeros(cache.k.shape[:2], dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        at = at_of(cache, b, n)
        touched[at] = True
        for name, new in (("k", k), ("v", v)):
            codes, scales = quantize_ref(new[b, L - n:])
            assert torch.equal(getattr(cache, name)[at], codes)
            assert torch.equal(getattr(cache, name + "_scales")[at], scales)
    for name, old in before.items():  # nothing else is written
        assert torch.equal(getattr(cache, name)[~touched], old[~touched])


def test_append_ties_extremes_and_blocks_that_are_not_finite(moe):  # noqa: F811
    D, vals = 128, [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.5, 7.98, 4.0, 0.0]
    rows = torch.zeros(9, D)
    for i, e in enumerate((0, 5, -20)):
        rows[i, :len(vals)] = torch.tensor(vals) * 2.0 ** e
        rows[i, 32:32 + len(vals)] = -torch.tensor(vals) * 2.0 ** e
        rows[i, 64] = -0.0
    rows[3, 7], rows[4, 40], rows[5, 100] = float("nan"), float("inf"), -float("inf")
    rows[3:6] += torch.arange(D) % 3 == 1
    rows[6, 0], rows[7, 1], rows[8, 2] = 3.3e38, 1e-38, -9.2e-41  # the largest block, and two at E8M0's lower end
    x = rows.to(BF).to(DEV)[None, :, None]
    cache, _ = make_cache(moe, [9], 1, D, 4)
    cache.append(x, x.flip(1).contiguous())
    cache.check()
    at = at_of(cache, 0, 9)
    for name, new in (("k", x), ("v", x.flip(1))):
        codes, scales = quantize_ref(new[0])
        assert torch.equal(getattr(cache, name)[at], codes) and torch.equal(getattr(cache, name + "_scales")[at], scales)
    assert set(cache.k_scales[at].flatten().tolist()) >= {255, 0, 252}


def test_append_skips_and_reports(moe):  # noqa: F811
    cache, g = make_cache(moe, [3, 9], 1, 64, 4, seed=8)
    k = randn(g, 2, 5, 1, 64).to(BF)
    cache.append(k, k)  # the first request's two oldest tokens have no place
    cache.check()
    assert torch.equal(cache.k[at_of(cache, 0, 3)], quantize_ref(k[0, 2:])[0])
    cache.block_table[1, 2] = cache.k.shape[0]
    cache.append(k, k)
    with pytest.raises(moe.MoEError, match="page index"):
        cache.check()


# ---------------------------------------------------------------------------------------------- attention
CASES = [  # lens, kv, group, L, D, page
    ([1], 1, 1, 1, 64, 1),
    ([0], 2, 4, 1, 128, 16),
    ([17, 0, 64, 65, 63], 2, 4, 1, 128, 16),
    ([333], 8, 4, 1, 128, 16),
    ([5, 130, 3, 0, 1000], 1, 16, 2, 64, 48),   # 32 rows; requests shorter than L
    ([2, 700, 8], 2, 4, 8, 128, 64),            # 32 rows, causal, fewer tokens than rows
    ([4000], 1, 7, 3, 128, 5),                  # 21 rows, odd pages
    ([260, 900], 2, 16, 4, 64, 16),             # 64 rows: two row tiles
    ([1200, 31], 1, 16, 5, 128, 33),            # 80 rows
    ([700, 90], 2, 4, 70, 64, 16),              # 280 rows, causal over several tiles
    ([30000], 1, 8, 1, 128, 128),               # one head spread over the whole GPU
    ([50] * 150, 1, 4, 1, 64, 16),              # many short units a block
    ([9] * 3 + [20000] + [1] * 300, 1, 2, 2, 64, 32),
]


@pytest.mark.parametrize("lens,kv,group,L,D,page", CASES)
def test_attend(moe, lens, kv, group, L, D, page):  # noqa: F811
    cache, g = make_cache(moe, lens, kv, D, page, seed=len(lens) + L)
    fill(cache, g, lens)
    q = (1.5 * randn(g, len(lens), L, kv * group, D)).to(BF)
    first = check_attend(cache, q, lens)
    again = check_attend(cache, q, lens)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("D,group,L", [(64, 2, 1), (128, 4, 6)])
@pytest.mark.parametrize("order", ["growing", "falling"])
def test_attend_large_scores_move_the_maximum(moe, D, group, L, order):  # noqa: F811
    """Scores that span hundreds of powers of two, in either order along the sequence."""
    n, kv = 700, 2
    cache, g = make_cache(moe, [n, 90], kv, D, 16, seed=5)
    k = randn(g, 2, n, kv, D)
    gain = torch.logspace(-2, 2, n, device=DEV)
    k = k * (gain if order == "growing" else gain.flip(0))[:, None, None]
    cache.append(k.to(BF), randn(g, 2, n, kv, D).to(BF))
    check_attend(cache, (2 * randn(g, 2, L, kv * group, D)).to(BF), [n, 90], scale=0.7)


def test_attend_strided_views_and_head_major_pages(moe):  # noqa: F811
    lens, kv, D, L, H = [70, 5, 400], 2, 128, 3, 8
    cache, g = make_cache(moe, lens, kv, D, 16, seed=9, layout="heads")
    fill(cache, g, lens)
    wide = randn(g, 3 * L, (H + 4) * D).to(BF)
    q = wide[:, :H * D].unflatten(0, (3, L)).unflatten(-1, (H, D))
    want, _ = check_attend(cache, q.contiguous(), lens)
    out = torch.full((3 * L, (H + 2) * D), 3.0, dtype=BF, device=DEV)
    cache.attend(q, out[:, D:(H + 1) * D].unflatten(0, (3, L)).unflatten(-1, (H, D)))
    assert torch.equal(out[:, D:(H + 1) * D].reshape(want.shape), want)
    assert torch.all(out[:, :D] == 3) and torch.all(out[:, (H + 1) * D:] == 3)


SCALES = [  # value scale bytes: inside fp16's exact range, at its ends, outside on either side, far apart, E8M0's ends
    (127, 127), (99, 135), (98, 127), (127, 136), (60, 120), (100, 200), (0, 0), (0, 127), (0, 3), (200, 225),
]


@pytest.mark.parametrize("D,group,L", [(64, 4, 2), (128, 8, 4)])
@pytest.mark.parametrize("lo,hi", SCALES)
def test_attend_values_of_any_scale(moe, D, group, L, lo, hi):  # noqa: F811
    lens, kv = [150, 20, 3], 2
    cache, g = make_cache(moe, lens, kv, D, 16, seed=lo + hi)
    fill(cache, g, lens)
    for b, n in enumerate(lens):
        at = at_of(cache, b, n)
        pick = torch.rand(cache.v_scales[at].shape, generator=g, device=DEV) < 0.5
        cache.v_scales[at] = torch.where(pick, lo, hi).to(torch.uint8)
    check_attend(cache, randn(g, 3, L, kv * group, D).to(BF), lens)


@pytest.mark.parametrize("D", [64, 128])
def test_attend_a_large_value_that_has_no_weight(moe, D):  # noqa: F811
    """A token whose value is 2^70 times the others' but whose weight is 0 must not take their digits."""
    n, kv = 200, 1
    cache, g = make_cache(moe, [n], kv, D, 16, seed=3)
    fill(cache, g, [n])
    at = at_of(cache, 0, n)
    cache.v_scales[at[0][77], at[1][77]] = 197
    cache.k_scales[at[0][77], at[1][77]] = 140
    cache.k[at[0][77], at[1][77]] = 0xFF  # all -6
    q = randn(g, 1, 2, 4, D).abs().to(BF)
    check_attend(cache, q, [n])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lo,hi", [(0, 0), (0, 4), (1, 226), (220, 226), (90, 160)])
def test_attend_keys_of_any_scale(moe, D, lo, hi):  # noqa: F811
    """Keys up to 2^99 and down to 2^-128, q scaled so that the scores stay moderate."""
    lens, kv = [150, 20], 2
    cache, g = make_cache(moe, lens, kv, D, 16, seed=lo + hi)
    fill(cache, g, lens)
    for b, n in enumerate(lens):
        at = at_of(cache, b, n)
        cache.k_scales[at] = torch.randint(lo, hi + 1, cache.k_scales[at].shape, generator=g, device=DEV).to(torch.uint8)
    top = 2.0 ** (127 - hi)
    q = (randn(g, 2, 2, 4, D) * min(top, 2.0 ** 120)).to(BF)
    check_attend(cache, q, lens, scale=1.0 if top < 2.0 ** 120 else 2.0 ** (127 - hi - 120))


@pytest.mark.parametrize("D,L", [(64, 1), (128, 1), (128, 5), (64, 40)])
def test_attend_nan_blocks_reach_only_the_rows_that_see_them(moe, D, L):  # noqa: F811
    n, kv, group = 130, 2, 4
    for which, hidden in (("k_scales", False), ("v_scales", False), ("k_scales", True), ("v_scales", True)):
        if hidden and L == 1:
            continue
        cache, g = make_cache(moe, [n, n], kv, D, 16, seed=L)
        fill(cache, g, [n, n])
        q = randn(g, 2, L, kv * group, D).to(BF)
        want, want_lse = (t.clone() for t in check_attend(cache, q, [n, n]))
        tok = n - 1 if hidden else 77  # the newest token is seen by the last row alone
        at = at_of(cache, 0, n)
        getattr(cache, which)[at[0][tok], at[1][tok], 1, 0] = 255  # head 1's first block
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
        cache.attend(q, out, lse)
        cache.check()
        first = max(L - n + tok, 0) if tok >= n - L else 0  # rows from here on see the token
        hit = torch.zeros(q.shape[:3], dtype=torch.bool, device=DEV)
        hit[0, first:, group:] = True
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
        if which == "k_scales":
            assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
        else:
            assert torch.isnan(out[hit][:, :32]).all() and torch.isfinite(out[hit][:, 32:]).all()
            assert torch.isfinite(lse[hit]).all()


def test_attend_q_that_is_not_finite(moe):  # noqa: F811
    n, kv, D = 90, 1, 128
    cache, g = make_cache(moe, [n], kv, D, 16)
    fill(cache, g, [n])
    q = randn(g, 1, 2, 4, D).to(BF)
    want = cache.attend(q).clone()
    q[0, 0, 1, 3], q[0, 1, 2, 100] = float("nan"), float("inf")
    out = cache.attend(q)
    hit = torch.zeros(1, 2, 4, dtype=torch.bool, device=DEV)
    hit[0, 0, 1] = hit[0, 1, 2] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], want[~hit])


@pytest.mark.parametrize("L", [1, 4])
def test_attend_many_tokens_of_small_weight(moe, L):  # noqa: F811
    """One token of large weight and 60,000 of 2^-24 each: what fp16 holds of the small weights must add up."""
    n, kv, D = 60001, 1, 64
    cache, g = make_cache(moe, [n], kv, D, 64)
    k = torch.zeros(1, n, kv, D, device=DEV)
    k[0, 500, 0, 0] = 6.0
    v = torch.ones(1, n, kv, D, device=DEV)
    v[0, 500] = -1
    cache.append(k.to(BF), v.to(BF))
    q = torch.zeros(1, L, 4, D, device=DEV)
    q[..., 0] = 4.0
    check_attend(cache, q.to(BF), [n], scale=math.log(2.0))


def test_attend_reports_bad_pages_and_lengths(moe):  # noqa: F811
    cache, g = make_cache(moe, [5, 90], 1, 64, 16, seed=8)
    fill(cache, g, [5, 90])
    q = randn(g, 2, 1, 4, 64).to(BF)
    cache.block_table[1, 2] = cache.k.shape[0]
    cache.attend(q)
    with pytest.raises(moe.MoEError, match="page index"):
        cache.check()
    cache.block_table[:] = 0
    cache.seq_lens[0] = -3
    cache.attend(q)
    with pytest.raises(moe.MoEError, match="sequence length"):
        cache.check()


def test_attend_between_other_formats_in_one_workspace(moe):  # noqa: F811
    """Row tiles, heads and grids of other sizes, in one workspace whose counters only are zero."""
    import test_gpu_decode as other
    calls, size = [], 0
    for i, (lens, kv, group, L, D, fmt) in enumerate([
            ([20000], 8, 4, 1, 128, "mxfp4"), ([300 + 17 * i for i in range(64)], 8, 4, 8, 128, "mxfp8"),
            ([300 + 17 * i for i in range(64)], 8, 4, 8, 128, "mxfp4"), ([4000, 9000], 2, 16, 4, 64, "mxfp4"),
            ([30000], 1, 8, 1, 128, "bf16"), ([30000], 1, 8, 1, 64, "mxfp4"), ([50] * 150, 1, 4, 1, 64, "mxfp4")]):
        src = make_cache(moe, lens, kv, D, 64, seed=i) if fmt == "mxfp4" else other.make_cache(moe, lens, kv, D, 64, fmt, seed=i)
        (fill if fmt == "mxfp4" else other.fill)(src[0], src[1], lens)
        q = (1.5 * randn(src[1], len(lens), L, kv * group, D)).to(BF)
        size = max(size, moe.lib().moe_paged_attention_workspace(src[0]._ref, kv * group, L))
        calls.append((src[0], q))
    ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    ws[:moe.MOE_ATTENTION_COUNTER_BYTES] = 0
    for cache, q in calls + calls[::-1]:
        n = moe.lib().moe_paged_attention_workspace(cache._ref, q.shape[2], q.shape[1])
        tail = ws[n:].clone()
        want = cache.attend(q, workspace=cache.attention_workspace(q.shape[2], q.shape[1]))
        got = cache.attend(q, workspace=ws[:n])
        assert torch.equal(got, want) and not torch.isnan(got).any()
        assert torch.all(ws[:moe.MOE_ATTENTION_COUNTER_BYTES] == 0) and torch.equal(ws[n:], tail)


def test_attend_and_append_in_a_graph(moe):  # noqa: F811
    lens, kv, D, L = [100, 7, 300], 2, 128, 2
    cache, g = make_cache(moe, lens, kv, D, 16, seed=21)
    fill(cache, g, lens)
    k, v, q = (randn(g, 3, L, h, D).to(BF) for h in (kv, kv, 8))
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.append(k, v)
        cache.attend(q, out)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            cache.append(k, v)
            cache.attend(q, out)
        for _ in range(2):
            k.normal_(generator=None)
            out.fill_(9)
            graph.replay()
        side.synchronize()
    ref, _, tol, _ = reference(cache, q, lens, D ** -0.5)
    assert torch.all((out.double() - ref).abs() <= tol)
