"""Head norms with the position rotation at the ends of what they allow, against plain implementations in 64 bits."""
import pytest
import torch

from test_gpu_decode import BF, DEV, gen, moe, randn  # noqa: F401
from test_gpu_rope import assert_rows, assert_stored, freqs, make, reference

pytestmark = pytest.mark.gpu

# heads whose squares leave fp32's range at either end (bf16's own is 9.2e-41 to 3.4e38), and ordinary ones between them
SIZES = [1.0, 3e36, 1e25, 1e19, 1e18, 1e-3, 1e-17, 1e-19, 1e-22, 1e-25, 1e-30, 1e-36, 1e-38, 1e-39, 0.03]


def heads_of_any_size(g, T, H, D):
    size = torch.tensor(SIZES, dtype=torch.float64, device=DEV)[torch.randint(0, len(SIZES), (T, H), generator=g, device=DEV)]
    x = (randn(g, T, H, D).double().clamp(-30, 30) * size[..., None]).to(BF)
    return torch.where((x == 0).all(-1, keepdim=True), torch.full_like(x, 2.0 ** -133), x)  # no head of zeros


@pytest.mark.parametrize("D,rot,pairs", [(128, 128, "half"), (64, 64, "adjacent"), (128, 50, "half"), (64, 0, "half")])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 2.0 ** -80, 1e-6, 2.0 ** 126])
def test_heads_whose_squares_leave_the_range(moe, D, rot, pairs, eps):  # noqa: F811
    T, g = 53, gen(D + rot)
    q, k = heads_of_any_size(g, T, 7, D), heads_of_any_size(g, T, 3, D)
    w = 1 + 0.3 * randn(g, D)
    plan = moe.RotaryPlan(freqs(rot), None, pairs, DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    out = moe.moe_head_norm_rope(q, k, plan, pos, w, w, eps)
    for got, x in zip(out, (q, k)):
        assert_rows(got, reference(x, w, eps, pos[None], freqs(rot), None, pairs))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
def test_keys_whose_squares_leave_the_range(moe, fmt):  # noqa: F811
    n, kv, D = 60, 3, 128
    cache, g = make(moe, fmt, [n], kv, D, 16, seed=1)
    k = heads_of_any_size(g, n, kv, D)
    w = 1 + 0.3 * randn(g, D)
    plan = moe.RotaryPlan(freqs(D), device=DEV)
    cache.append_rotated(None, k[None], k[None], plan, None, None, w, 0.0)
    cache.check()
    assert_stored(fmt, cache, 0, n, "k", reference(k, w, 0.0, torch.arange(n, device=DEV)[None], freqs(D), None, "half"))


def test_heads_that_are_not_finite_keep_to_themselves(moe):  # noqa: F811
    """A NaN makes its head NaN, an infinity is NaN among zeros (x / inf); large heads beside them are not touched."""
    D = 64
    x = torch.full((2, 4, D), 3e38, device=DEV).to(BF)
    x[0, 1, 7], x[1, 2, 9], x[1, 3, 0] = float("nan"), float("inf"), -float("inf")
    y = moe.moe_head_norm_rope(x, None, moe.RotaryPlan([], device=DEV), None, torch.ones(D, device=DEV), eps=1e-6)[0]
    want = torch.ones_like(x)
    want[0, 1], want[1, 2], want[1, 3] = float("nan"), 0, 0
    want[1, 2, 9] = want[1, 3, 0] = float("nan")
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(y.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
def test_on_another_stream(moe, fmt):  # noqa: F811
    """Outputs of a call on a stream of its own, read after that stream: what the call gives on the current one, bit for bit."""
    lens, L, kv, D = [200, 3, 50], 2, 2, 128
    cache, g = make(moe, fmt, lens, kv, D, 16, seed=4)
    other = make(moe, fmt, lens, kv, D, 16, seed=4)[0]
    q, k, v = randn(g, len(lens), L, 8, D).to(BF).split((4, 2, 2), dim=2)
    plan, w = moe.RotaryPlan(freqs(D), device=DEV), torch.ones(D, device=DEV)
    want = cache.append_rotated(q, k, v, plan, None, w, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [other.append_rotated(q, k, v, plan, None, w, w, stream=side)]
    got += moe.moe_head_norm_rope(q, k, plan, (other.seq_lens[:, None] - L + torch.arange(L, device=DEV)).int(), w, w)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], want)
    for n in ("k", "v") + (("k_scales", "v_scales") if fmt != "bf16" else ()):
        assert torch.equal(getattr(other, n).view(torch.uint8), getattr(cache, n).view(torch.uint8))
