"""The attention over a 4-bit cache where a block works through many units one after another: whole ones, and parts of shared
ones that it joins right before it begins the next."""
import pytest
import torch

import test_gpu_cache_fp4 as fp4
from test_gpu_decode import BF, DEV, gen, moe, randn  # noqa: F401

pytestmark = pytest.mark.gpu

MIXED = [3000, 1, 40, 900, 0, 2, 2500, 130, 7, 64] * 6
SHORT = [1, 33, 0, 128, 5, 129, 64] * 40


@pytest.mark.parametrize("lens,kv,group,L,D,page", [
    (MIXED, 4, 4, 1, 128, 64),     # 8 rows a head (and so on below: every row tile that there is)
    (SHORT, 4, 4, 1, 128, 16),
    (MIXED, 4, 2, 8, 128, 16),     # 16
    (SHORT, 4, 4, 6, 128, 16),     # 24
    (MIXED, 4, 4, 8, 128, 64),     # 32
    (SHORT, 4, 4, 8, 128, 16),
    (SHORT[:140], 2, 8, 9, 128, 16),  # 72: three row tiles a head
    (MIXED, 4, 8, 1, 64, 64),
    (SHORT, 4, 8, 2, 64, 16),
    (MIXED, 4, 8, 3, 64, 48),
    (SHORT, 4, 8, 4, 64, 16),
    (MIXED, 4, 8, 6, 64, 64),      # 48
    (SHORT, 4, 8, 5, 64, 16),
])
def test_rows_go_to_their_own_unit(moe, lens, kv, group, L, D, page):  # noqa: F811
    """A warp that begins the next unit while another still writes the last one's rows must not hand it that unit's places: every
    row has values of its own, outputs are poisoned before every run, and all runs give the first one's bits."""
    cache, g = fp4.make_cache(moe, lens, kv, D, page, seed=len(lens) + L)
    fp4.fill(cache, g, lens)
    q = (1.5 * randn(g, len(lens), L, kv * group, D)).to(BF)
    out, lse = fp4.check_attend(cache, q, lens)
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    for _ in range(40):
        again.fill_(float("nan"))
        lse2.fill_(float("nan"))
        cache.attend(q, again, lse2)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    cache.check()


@pytest.mark.parametrize("lens,kv,group,L,D,page", [
    ([15000], 3, 2, 1, 64, 16),          # three heads side by side, one unit over 152 blocks of each
    ([9000, 5, 0, 700], 17, 1, 2, 64, 16),   # 17 has no divisor up to 16: heads one after another, joins in two steps
    ([12000], 18, 2, 1, 128, 64),        # two groups of nine heads: 304 or 456 blocks leave some without work
    ([12000, 77], 18, 2, 3, 64, 48),
    ([6000, 1, 300], 32, 2, 1, 128, 16),     # two groups of 16
    (SHORT[:35], 32, 1, 5, 64, 16),
    ([40] * 60 + [4000], 24, 2, 4, 64, 16),  # two of twelve, several short units a block
    ([3000, 0, 129], 33, 3, 8, 128, 64),     # three of eleven, 24 rows a head
    ([500, 64], 65, 1, 20, 64, 16),          # five of thirteen
    ([2000], 48, 1, 70, 64, 16),             # three of 16, three row tiles
])
def test_heads_in_groups(moe, lens, kv, group, L, D, page):  # noqa: F811
    """Blocks read up to 16 key-value heads side by side, the largest number that divides them; the other heads follow."""
    cache, g = fp4.make_cache(moe, lens, kv, D, page, seed=kv + L)
    fp4.fill(cache, g, lens)
    q = (1.5 * randn(g, len(lens), L, kv * group, D)).to(BF)
    out, lse = fp4.check_attend(cache, q, lens)
    again = fp4.check_attend(cache, q, lens)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("D,group,L", [(128, 4, 1), (64, 8, 4)])
@pytest.mark.parametrize("gap", [8, 15, 19, 22, 27, 33])
def test_weights_far_below_the_largest(moe, D, group, L, gap):  # noqa: F811
    """One token, whose values are zeros, takes nearly all weight; the others hold 2^-gap of it each.  fp16 keeps eleven bits of
    them down to a gap of 20 and an error of 2^-31 of the largest below; lse keeps them all."""
    n, kv = 3000, 2
    cache, g = fp4.make_cache(moe, [n], kv, D, 64, seed=gap)
    k, v = 0.25 * randn(g, 1, n, kv, D), randn(g, 1, n, kv, D).abs()
    k[..., 0], v[:, 100] = 0, 0
    k[:, 100] = 0
    k[:, 100, :, 0] = 4.0
    cache.append(k.to(BF), v.to(BF))
    q = 0.25 * randn(g, 1, L, kv * group, D)
    q[..., 0] = gap * 0.6931 / (4.0 * D ** -0.5)
    q = q.to(BF)
    out, _ = fp4.check_attend(cache, q, [n])
    if gap <= 19:  # of sums of positive values nothing but roundings is lost: 2^-8 of out, 2^-11 of a weight, 2^-9 for scores
        ref = fp4.reference(cache, q, [n], D ** -0.5)[0]
        assert torch.all((out.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -9) * ref)
    if gap == 33:
        assert torch.all(out.abs() <= 3000 * 2.0 ** -31 * 4)
