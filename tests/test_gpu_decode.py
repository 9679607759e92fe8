"""The decode-step operators on the GPU against plain implementations in 64 bits: the residual addition with its
norm, the paged cache's writer and the attention that reads it."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
HALF_ULP = 2.0 ** -8  # bf16: half a unit in the last place, relative to the value


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__ as g
    g.build_cuda()
    import block_scaled_fp4_sqrt_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def mxfp8_ref(x_bf16: torch.Tensor):
    """(codes, scale bytes) of bf16 rows by the oracle's quantiser."""
    rows = x_bf16.reshape(-1, x_bf16.shape[-1])
    bits = np.ascontiguousarray(rows.cpu().view(torch.int16).numpy().view(np.uint16))
    q, s = oracle.quantize_x(bits)
    return torch.from_numpy(np.asarray(q)).reshape(x_bf16.shape), torch.from_numpy(np.asarray(s)).reshape(
        *x_bf16.shape[:-1], -1)


# ---------------------------------------------------------------------------------------------- norm
def norm_ref(x, r, w, eps):
    t = x.double() + (0 if r is None else r.double())
    return t, t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps) * w.double()


def assert_norm_y(y, ref):
    # one rounding to bf16, and fp32 sums of up to 65536 squares in blocks: below 2^-17 relative
    assert torch.all((y.double() - ref).abs() <= (HALF_ULP + 2.0 ** -17) * ref.abs() + 1e-37)


@pytest.mark.parametrize("T,d", [(1, 8), (3, 40), (9, 512), (1, 520), (5, 1024), (7, 4096), (300, 2560), (2, 16384),
                                 (2, 16392), (3, 32768), (2, 65536)])
@pytest.mark.parametrize("with_r,w32", [(True, False), (False, True)])
def test_norm(moe, T, d, with_r, w32):
    g = gen(T * 70001 + d)
    x, r = (4 * randn(g, T, d)).to(BF), (randn(g, T, d)).to(BF) if with_r else None
    w = 1 + 0.3 * randn(g, d)
    w = w if w32 else w.to(BF)
    s, y = torch.full((T, d), 9.0, dtype=BF, device=DEV), torch.full((T, d), 9.0, dtype=BF, device=DEV)
    mx = d % 32 == 0
    yq = torch.empty(T, d, dtype=torch.uint8, device=DEV) if mx else None
    ys = torch.empty(T, d // 32, dtype=torch.uint8, device=DEV) if mx else None
    moe.moe_add_rms_norm(x, r, w, 1e-5, s, y, yq, ys)
    t, ref = norm_ref(x, r, w, 1e-5)
    assert torch.equal(s, (x.float() + (0 if r is None else r.float())).to(BF))
    assert_norm_y(y, ref)
    if mx:
        q0, s0 = mxfp8_ref(y)
        assert torch.equal(yq.cpu(), q0) and torch.equal(ys.cpu(), s0)


def test_norm_zero_rows_and_extremes(moe):
    d = 256
    x = torch.zeros(4, d, dtype=BF, device=DEV)
    x[1] = 1e-20
    x[2, 5] = 3e18  # its square is within fp32
    x[3] = -1e-3
    w = torch.ones(d, device=DEV)
    y = torch.empty_like(x)
    yq, ys = torch.empty(4, d, dtype=torch.uint8, device=DEV), torch.empty(4, d // 32, dtype=torch.uint8, device=DEV)
    moe.moe_add_rms_norm(x, None, w, 1e-6, None, y, yq, ys)
    assert_norm_y(y, norm_ref(x, None, w, 1e-6)[1])
    assert torch.all(y[0] == 0) and torch.all(ys[0] == 0) and torch.all(yq[0] == 0)


def test_norm_nan_stays_in_its_row(moe):
    x = torch.ones(3, 64, dtype=BF, device=DEV)
    x[1, 7] = float("nan")
    y = torch.empty_like(x)
    moe.moe_add_rms_norm(x, None, torch.ones(64, device=DEV), 0.0, None, y)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2]).all()


def test_norm_strides_in_place_and_single_outputs(moe):
    g = gen(5)
    T, d = 33, 1536
    wide = randn(g, T, 2 * d + 8).to(BF)
    x, r = wide[:, :d], wide[:, d + 8:]  # both row-strided
    w = randn(g, d).to(BF)
    want = (x.float() + r.float()).to(BF)
    ref = norm_ref(x, r, w, 1e-6)[1]
    out = torch.zeros(T, d + 64, dtype=BF, device=DEV)
    moe.moe_add_rms_norm(x, r, w, 1e-6, None, out[:, :d])
    assert_norm_y(out[:, :d], ref)
    assert torch.all(out[:, d:] == 0)
    moe.moe_add_rms_norm(x, r, w, 1e-6, r, x)  # the stream in place, the norm over x
    assert torch.equal(r, want)
    assert_norm_y(x, ref)
    moe.moe_add_rms_norm(torch.empty(0, d, dtype=BF, device=DEV), None, w, 1e-6, None, torch.empty(0, d, dtype=BF, device=DEV))


def test_norm_mxfp8_feeds_the_expert_ffn_like_permute(moe):
    """y_q / y_s are the bytes moe_permute writes for y."""
    from gpu_support import case
    wl, inp, ids, wts, layer = case("tiny")
    g = gen(11)
    x, r, w = randn(g, wl.T, wl.d).to(BF), randn(g, wl.T, wl.d).to(BF), torch.ones(wl.d, device=DEV)
    y = torch.empty_like(x)
    yq = torch.empty(wl.T, wl.d, dtype=torch.uint8, device=DEV)
    ys = torch.empty(wl.T, wl.d // 32, dtype=torch.uint8, device=DEV)
    moe.moe_add_rms_norm(x, r, w, 1e-6, None, y, yq, ys)
    p = layer.permute(y, torch.from_numpy(ids).to(DEV))
    perm = p["perm_tok"].long()
    assert torch.equal(p["a_q"], yq[perm]) and torch.equal(p["a_s"], ys[perm])


# ---------------------------------------------------------------------------------------------- cache
def make_cache(moe, lens, kv, D, page, fmt, seed=0, layout="rows", spare=2, first_page=0, n_pages=None):
    """A cache of random contents whose unused rows hold NaN; pages of the requests in random order."""
    g = gen(seed)
    lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    per = [-(-n // page) for n in lens]
    need = sum(per)
    n_pages = n_pages or need + spare
    perm = (torch.randperm(n_pages - first_page, generator=g, device=DEV) + first_page).tolist()
    table = torch.full((len(lens), max(per + [1]) + 1), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    table = table.to(DEV)
    shape = (n_pages, page, kv, D)
    inner = (n_pages, kv, page, D) if layout == "heads" else shape
    fix = (lambda t: t.transpose(1, 2)) if layout == "heads" else (lambda t: t)
    if fmt == "bf16":
        k, v = (fix(torch.full(inner, float("nan"), dtype=BF, device=DEV)) for _ in "kv")
        sc = (None, None)
    else:
        k, v = (fix(torch.full(inner, 0x7F, dtype=torch.uint8, device=DEV)) for _ in "kv")
        sc = tuple(fix(torch.full((*inner[:3], D // 32), 200, dtype=torch.uint8, device=DEV)) for _ in "kv")
    cache = moe.PagedKVCache(k, v, table, lens_t, *sc)
    cache.tab = table.cpu()
    return cache, g


def rows_of(cache, b, n, which):
    """Request b's first n rows as fp64 [n, kv, D]."""
    pages = getattr(cache, which)
    sc = getattr(cache, which + "_scales")
    page = pages.shape[1]
    pos = torch.arange(n)
    at = (cache.tab[b, pos // page].long().to(DEV), (pos % page).to(DEV))
    r = pages[at]
    if sc is None:
        return r.double()
    e = sc[at].double() - 127
    return (r.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32)) * torch.exp2(e)[..., None]).flatten(-2)


def fill(cache, g, lens, k_gain=1.0):
    """Append the whole context of every request at once; returns the bf16 keys and values."""
    L = max(lens)
    if L == 0:
        return None, None
    k = (k_gain * randn(g, len(lens), L, cache.n_kv_heads, cache.head_dim)).to(BF)
    v = randn(g, len(lens), L, cache.n_kv_heads, cache.head_dim).to(BF)
    cache.append(k, v)
    return k, v


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("lens,kv,D,page", [([1], 1, 64, 1), ([0, 5, 64, 65], 2, 128, 16), ([7, 300, 2], 3, 64, 48),
                                            ([129], 8, 128, 3)])
def test_append_writes_every_token_exactly(moe, fmt, lens, kv, D, page):
    cache, g = make_cache(moe, lens, kv, D, page, fmt, seed=sum(lens))
    before = {n: getattr(cache, n).clone() for n in ("k", "v")}
    k, v = fill(cache, g, lens)
    L = max(lens)
    cache.check()
    touched = torch.zeros(cache.k.shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens):
        for i in range(n):
            touched[cache.tab[b, i // page], i % page] = True
        if n == 0:
            continue
        for name, new in (("k", k), ("v", v)):
            want = new[b, L - n:]
            pos = torch.arange(n)
            at = (cache.tab[b, pos // page].long().to(DEV), (pos % page).to(DEV))
            if fmt == "bf16":
                assert torch.equal(getattr(cache, name)[at], want)
            else:
                q, s = mxfp8_ref(want.contiguous())
                assert torch.equal(getattr(cache, name)[at].cpu(), q)
                assert torch.equal(getattr(cache, name + "_scales")[at].cpu(), s)
    for name in ("k", "v"):  # nothing else is written
        a, b = getattr(cache, name).cpu()[~touched], before[name].cpu()[~touched]
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_append_a_step_from_a_fused_projection(moe, fmt):
    lens, kv, D, L = [3, 40, 0, 129, 4], 2, 128, 4
    cache, g = make_cache(moe, lens, kv, D, 32, fmt, seed=3, layout="heads")
    fill(cache, g, lens)
    qkv = randn(g, len(lens) * L, 8 * D + 2 * kv * D).to(BF)
    k = qkv[:, 8 * D:8 * D + kv * D].unflatten(0, (len(lens), L)).unflatten(-1, (kv, D))
    v = qkv[:, 8 * D + kv * D:].unflatten(0, (len(lens), L)).unflatten(-1, (kv, D))
    cache.append(k, v)
    cache.check()
    for b, n in enumerate(lens):
        for name, new in (("k", k), ("v", v)):
            got = rows_of(cache, b, n, name)
            m = min(n, L)
            if m == 0:
                continue
            want = new[b, L - m:].contiguous()
            if fmt == "mxfp8":
                q, s = mxfp8_ref(want)
                want = (q.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32)) *
                        torch.exp2(s.double() - 127)[..., None]).flatten(-2).to(DEV)
            assert torch.equal(got[n - m:], want.double())


def test_append_reports_bad_pages_and_lengths(moe):
    cache, g = make_cache(moe, [5, 9], 1, 64, 4, "bf16", seed=8)
    cache.block_table[1, 2] = cache.k.shape[0]  # one past the last page
    k = randn(g, 2, 2, 1, 64).to(BF)
    cache.append(k, k)
    with pytest.raises(moe.MoEError, match="page index"):
        cache.check()
    cache.check()
    cache.seq_lens[0] = cache.block_table.shape[1] * 4 + 1
    cache.block_table[:] = 0
    cache.append(k, k)
    with pytest.raises(moe.MoEError, match="sequence length"):
        cache.check()


# ---------------------------------------------------------------------------------------------- attention
def attend_ref(cache, q, lens, scale):
    """out, lse in 64 bits, and the error bounds that go with them.

    Scores: the products are exact, their fp32 sum of D terms errs by at most D 2^-24 sum |q k|; an MXFP8 cache's
    split of q adds at most 2^-17 max|q| per term.  p and z carry that relative error and 2^-20 more for the
    exponential and the fp32 sums; p is rounded to bf16 (2^-8 at most), the output once more."""
    B, L, H, D = q.shape
    kv = cache.n_kv_heads
    gsz = H // kv
    out = torch.zeros(B, L, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, L, H), -math.inf, dtype=torch.float64, device=DEV)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        K, V = rows_of(cache, b, n, "k"), rows_of(cache, b, n, "v")
        for l in range(L):
            end = n - L + 1 + l
            if end <= 0:
                continue
            qq = q[b, l].double().reshape(kv, gsz, D)
            s = torch.einsum("hgd,thd->hgt", qq, K[:end]) * scale
            mag = torch.einsum("hgd,thd->hgt", qq.abs(), K[:end].abs())
            err = D * 2.0 ** -24 * mag
            if cache.k_scales is not None:
                err = err + 2.0 ** -17 * qq.abs().amax(-1)[..., None] * K[:end].abs().sum(-1).t()[:, None, :]
            err = (abs(scale) * err).amax(-1) + 2.0 ** -20
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[..., None])
            lse[b, l] = z.reshape(-1)
            o = torch.einsum("hgt,thd->hgd", p, V[:end])
            out[b, l] = o.reshape(H, D)
            a = torch.einsum("hgt,thd->hgd", p, V[:end].abs())
            tol[b, l] = (HALF_ULP * o.abs() * 1.01 + (HALF_ULP * 1.01 + 2 * err[..., None]) * a + 1e-30).reshape(H, D)
            tol_lse[b, l] = (err + 2.0 ** -21 * z.abs()).reshape(-1)
    return out, lse, tol, tol_lse


def check_attend(cache, q, lens, scale=None, **kw):
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    out = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
    got = cache.attend(q, out, lse, scale, **kw)
    assert got is out
    torch.cuda.synchronize()
    cache.check()
    ref, rl, tol, tl = attend_ref(cache, q, lens, q.shape[-1] ** -0.5 if scale is None else scale)
    err = (out.double() - ref).abs()
    assert torch.all(err <= tol), f"out: {float((err - tol).max()):.3e} above its bound"
    dead = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), dead) and torch.all(out[dead] == 0)
    el = (lse.double() - rl).abs()[~dead]
    assert torch.all(el <= tl[~dead]), f"lse: {float((el - tl[~dead]).max()):.3e} above its bound"
    return out, lse


CASES = [  # lens, kv, group, L, D, page
    ([1], 1, 1, 1, 64, 1),
    ([0], 2, 4, 1, 128, 16),
    ([17, 0, 64, 65, 63], 2, 4, 1, 128, 16),
    ([333], 8, 4, 1, 128, 16),
    ([5, 130, 3, 0, 1000], 1, 16, 2, 64, 48),   # 32 rows; requests shorter than L
    ([2, 700, 8], 2, 4, 8, 128, 64),            # 32 rows, causal, fewer tokens than rows
    ([4000], 1, 7, 3, 128, 5),                  # 21 rows, odd pages
    ([260, 900], 2, 16, 4, 64, 16),             # 64 rows
    ([1200, 31], 1, 16, 5, 128, 33),            # 80 rows: two row tiles
    ([30000], 1, 8, 1, 128, 128),               # one head spread over the whole GPU
    ([50] * 150, 1, 4, 1, 64, 16),              # many short units a block
    ([9] * 3 + [20000] + [1] * 300, 1, 2, 2, 64, 32),
]


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("lens,kv,group,L,D,page", CASES)
def test_attend(moe, fmt, lens, kv, group, L, D, page):
    cache, g = make_cache(moe, lens, kv, D, page, fmt, seed=len(lens) + L)
    fill(cache, g, lens)
    q = (1.5 * randn(g, len(lens), L, kv * group, D)).to(BF)
    out, lse = check_attend(cache, q, lens)
    again = cache.attend(q)  # same bits, and the counters of the first call were left ready
    assert torch.equal(again, out)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_attend_strides_layouts_and_streams(moe, fmt):
    lens, kv, group, L, D = [70, 500], 2, 4, 2, 128
    cache, g = make_cache(moe, lens, kv, D, 16, fmt, seed=21, layout="heads")
    fill(cache, g, lens)
    H = kv * group
    qkv = randn(g, len(lens) * L, (H + 2 * kv) * D).to(BF)
    q = qkv[:, :H * D].unflatten(0, (len(lens), L)).unflatten(-1, (H, D))
    want, _ = check_attend(cache, q, lens, scale=-0.2)
    wide = torch.full((len(lens) * L, H * D + 16), 3.0, dtype=BF, device=DEV)
    out = wide[:, :H * D].unflatten(0, (len(lens), L)).unflatten(-1, (H, D))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.attend(q, out, scale=-0.2, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.all(wide[:, H * D:] == 3.0)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_attend_peaked_and_extreme_scores(moe, fmt):
    """Scores in the hundreds (one key takes all), keys all alike, and rows of zero queries."""
    lens, D = [1000, 200], 64
    cache, g = make_cache(moe, lens, 1, D, 16, fmt, seed=31)
    fill(cache, g, lens, k_gain=30.0)
    q = (10 * randn(g, 2, 1, 4, D)).to(BF)
    q[1, 0, 2] = 0
    q[1, 0, 3] *= 1e-30
    check_attend(cache, q, lens)


def test_attend_scales_across_the_e8m0_range(moe):
    """MXFP8 caches whose blocks lie far from 1: the packed multiplier, and above 2^7 its second factor."""
    lens, D = [100], 128
    for k_exp, v_exp in ((-40, 0), (0, 30), (0, -60), (12, 12), (-3, 8)):
        cache, g = make_cache(moe, lens, 1, D, 16, "mxfp8", seed=41)
        k = (randn(g, 1, 100, 1, D) * 2.0 ** k_exp).to(BF)
        v = (randn(g, 1, 100, 1, D) * 2.0 ** v_exp).to(BF)
        v[0, ::3] *= 2.0 ** 9
        cache.append(k, v)
        q = (randn(g, 1, 1, 4, D) * 2.0 ** -k_exp).to(BF)
        check_attend(cache, q, lens)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attend_rows_do_not_see_later_tokens_whatever_they_hold(moe, fmt, bad):
    lens, kv, group, L, D = [90, 6], 1, 4, 4, 64
    cache, g = make_cache(moe, lens, kv, D, 16, fmt, seed=51)
    fill(cache, g, lens)
    q = randn(g, 2, L, kv * group, D).to(BF)
    want = cache.attend(q).clone()
    for b, n in enumerate(lens):
        page, row = int(cache.tab[b, (n - 2) // 16]), (n - 2) % 16  # the token that rows 0, 1 don't see
        for pages in (cache.k, cache.v):
            if fmt == "bf16":
                pages[page, row] = bad
            else:
                pages[page, row] = 0x7F  # NaN: E4M3 has no infinity
    got = cache.attend(q)
    # the rows before the token are computed by other instructions, to the same bounds
    cache_ok = torch.allclose(got[:, :2].float(), want[:, :2].float(), rtol=2 * HALF_ULP, atol=2 * HALF_ULP)
    assert cache_ok and torch.isfinite(got[:, :2]).all()
    assert torch.isnan(got[:, 2:]).all()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_attend_far_offsets(moe, fmt):
    """Pages beyond 2^32 bytes (and 2^31 elements) into the pool."""
    D, page, kv = 128, 64, 8
    n_pages = (2 ** 32) // (page * kv * D) + 40
    cache, g = make_cache(moe, [1500], kv, D, page, fmt, seed=61, first_page=n_pages - 30, n_pages=n_pages)
    fill(cache, g, [1500])
    q = randn(g, 1, 1, kv * 2, D).to(BF)
    check_attend(cache, q, [1500])


def test_attend_shared_prefix_and_changing_lengths_in_a_graph(moe):
    kv, group, D, page = 2, 4, 128, 16
    cache, g = make_cache(moe, [256, 256], kv, D, page, "bf16", seed=71)
    fill(cache, g, [256, 256])
    cache.block_table[1, :4] = cache.block_table[0, :4]  # one prompt of 64 tokens, kept once
    cache.tab = cache.block_table.cpu()
    k, v = (randn(g, 2, 1, kv, D).to(BF) for _ in "kv")
    q = randn(g, 2, 1, kv * group, D).to(BF)
    cache.seq_lens.copy_(torch.tensor([65, 65], dtype=torch.int32))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        out = torch.empty_like(q)
        cache.append(k, v)
        cache.attend(q, out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            cache.append(k, v)
            cache.attend(q, out)
    for n in ([66, 100], [200, 65]):
        k.copy_(randn(g, 2, 1, kv, D))
        cache.seq_lens.copy_(torch.tensor(n, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref, _, tol, _ = attend_ref(cache, q, n, D ** -0.5)
        assert torch.all((out.double() - ref).abs() <= tol)


def test_attend_bad_page_is_reported_and_not_read(moe):
    cache, g = make_cache(moe, [100, 50], 1, 64, 16, "bf16", seed=81)
    fill(cache, g, [100, 50])
    q = randn(g, 2, 1, 2, 64).to(BF)
    want = cache.attend(q).clone()
    cache.block_table[0, 3] = 10 ** 6
    got = cache.attend(q)
    with pytest.raises(moe.MoEError, match="page index"):
        cache.check()
    assert torch.equal(got[1], want[1])


def test_attend_empty_calls(moe):
    cache, _ = make_cache(moe, [5], 1, 64, 16, "bf16")
    assert cache.attend(torch.empty(1, 0, 2, 64, dtype=BF, device=DEV)).shape == (1, 0, 2, 64)
    none = moe.PagedKVCache(cache.k, cache.v, torch.empty(0, 3, dtype=torch.int32, device=DEV),
                            torch.empty(0, dtype=torch.int32, device=DEV))
    assert none.attend(torch.empty(0, 2, 2, 64, dtype=BF, device=DEV)).shape == (0, 2, 2, 64)
    none.append(*(torch.empty(0, 2, 1, 64, dtype=BF, device=DEV) for _ in "kv"))


@pytest.mark.parametrize("fmt,D", [("bf16", 64), ("mxfp8", 64), ("mxfp8", 128)])
@pytest.mark.parametrize("L", [1, 3])
def test_attend_a_nan_value_reaches_the_rows_that_see_it(moe, fmt, D, L):
    """A NaN among the values of an old token, in one column: that column of its head is NaN, the others are not."""
    lens, kv, group = [150, 40], 2, 2
    cache, g = make_cache(moe, lens, kv, D, 16, fmt, seed=91)
    fill(cache, g, lens)
    q = randn(g, 2, L, kv * group, D).to(BF)
    want = cache.attend(q).clone()
    page, col = int(cache.tab[0, 70 // 16]), D // 2 + 5
    cache.v[page, 70 % 16, 1, col] = float("nan") if fmt == "bf16" else 0xFF
    got = cache.attend(q)
    assert torch.isnan(got[0, :, group:, col]).all()
    got[0, :, group:, col] = want[0, :, group:, col]
    # the tile with the NaN may be computed by other instructions, to the same bounds
    assert torch.allclose(got.float(), want.float(), rtol=2 * HALF_ULP, atol=2 * HALF_ULP)


@pytest.mark.parametrize("D", [64, 128])
def test_attend_a_later_token_of_the_largest_scale_stays_out(moe, D):
    """448 2^127 leaves bf16's range: a token that a row does not see must not turn the row into 0 times infinity."""
    lens, kv, group, L = [90], 1, 2, 3
    cache, g = make_cache(moe, lens, kv, D, 16, "mxfp8", seed=95)
    fill(cache, g, lens)
    q = randn(g, 1, L, kv * group, D).to(BF)
    want = cache.attend(q).clone()
    page, row = int(cache.tab[0, 89 // 16]), 89 % 16  # seen by the last row alone
    cache.v[page, row] = 0x7E
    cache.v_scales[page, row] = 254
    got = cache.attend(q)
    assert torch.allclose(got[:, :2].float(), want[:, :2].float(), rtol=2 * HALF_ULP, atol=2 * HALF_ULP)


def test_append_more_rows_than_one_launch_takes(moe):
    """2^27 and some tokens of a head of 64 (17 GB of keys): beyond 2^30 units the call goes on in a second launch."""
    L, D, page = 2 ** 27 + 1003, 64, 2 ** 20
    n_pages = -(-L // page)
    bits = torch.arange(L * D // 4, dtype=torch.int64, device=DEV) * 0x0001000300050007  # four columns, none alike
    new = bits.view(BF).view(1, L, 1, D)
    table = torch.arange(n_pages, dtype=torch.int32, device=DEV).flip(0).reshape(1, -1).contiguous()
    cache = moe.PagedKVCache(*(torch.zeros(n_pages, page, 1, D, dtype=BF, device=DEV) for _ in "kv"), table,
                             torch.tensor([L], dtype=torch.int32, device=DEV))
    cache.append(new, new)
    cache.check()
    rows = new.view(torch.int16).view(L, D)
    for pages in (cache.k, cache.v):
        for j in range(n_pages):
            n = min(page, L - j * page)
            assert torch.equal(pages[n_pages - 1 - j, :n, 0].view(torch.int16), rows[j * page:j * page + n])
