"""The decode-step operators run together (examples/decode_block.py), step after step, against the same block in
64 bits."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    import __graft_entry__ as g
    g.build_cuda()
    import decode_block
    return decode_block


def norm64(t, w, eps):
    return t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps) * w.double()


def attend64(q, k, v, n_new):
    """q [L, hq, D], k, v [n, hk, D] in fp64: causal among the L newest."""
    group, n = q.shape[1] // k.shape[1], k.shape[0]
    s = torch.einsum("lhd,thd->lht", q, k.repeat_interleave(group, 1)) * q.shape[-1] ** -0.5
    seen = torch.arange(n, device=DEV)[None, :] < (n - n_new + 1 + torch.arange(n_new, device=DEV))[:, None]
    p = torch.softmax(s.masked_fill(~seen[:, None, :], float("-inf")), -1)
    return torch.einsum("lht,thd->lhd", p, v.repeat_interleave(group, 1))


@pytest.mark.parametrize("B,L", [(1, 1), (2, 2), (3, 4)])  # 1 and 4 rows: forward_few; 12: forward
def test_steps_match_the_block_in_64_bits(example, B, L):
    """What the block hands from call to call is compared at each hand-over: the cache's rows and the attention at the
    bf16 roundings of their own inputs, the residual stream after the attention at the roundings of the whole half."""
    d, n_q, n_kv, hd, steps = 512, 8, 2, 64, 5
    block = example.random_block(d, 256, 8, 2, n_q, n_kv, hd, B, 64, L, page=16, fmt="bf16", seed=B)
    g = torch.Generator(device=DEV).manual_seed(77)
    ks, vs = [], []
    for i in range(steps):
        x = torch.randn(B * L, d, device=DEV, generator=g).to(BF)
        res = torch.randn(B * L, d, device=DEV, generator=g).to(BF)
        block.cache.seq_lens.add_(L)
        out, stream = block.step(x, res, L)
        block.cache.check()
        block.layer.check()
        t = x.double() + res.double()
        y = norm64(t, block.norm_attn, block.eps)
        qkv = (y @ block.w_qkv.double().t()).view(B, L, n_q + 2 * n_kv, hd)
        q, k, v = qkv.split((n_q, n_kv, n_kv), dim=2)
        ks.append(k)
        vs.append(v)
        o = torch.stack([attend64(q[b], torch.cat([c[b] for c in ks]), torch.cat([c[b] for c in vs]), L)
                         for b in range(B)])
        ref = t + o.reshape(B * L, -1) @ block.w_o.double().t()
        # y, q, k, v, p, o, the projection and the stream are each rounded to bf16 (2^-9 of the value): the scores are
        # of order 1, so an error of 2^-9 sqrt(2) of them moves p by as much; ten such roundings, five deviations
        # of their root sum of squares, relative to the stream's rms
        rms = ref.square().mean().sqrt()
        assert (stream.double() - ref).abs().max() <= 5 * 10 ** 0.5 * 2.0 ** -9 * rms * 2
        # the MoE half: both forms of the layer on the very rows that the block hands over
        y2 = torch.empty_like(x)
        example.moe.moe_add_rms_norm(stream, None, block.norm_moe, block.eps, y=y2)
        again = block.layer.forward(y2)
        assert out.shape == again.shape and torch.isfinite(out.double()).all()
        # y2 comes from the rounded stream here: a row's norm differs by roundings, and a routing decision may differ
        # between experts of equal score; the layer's outputs agree row by row except there
        err = (out.double() - again.double()).square().mean(-1).sqrt()
        assert (err <= 0.1 * again.double().square().mean(-1).sqrt()).double().mean() >= 0.5


def test_a_captured_step_replays_as_it_ran(example):
    B, L, d = 2, 2, 512
    args = (d, 256, 8, 2, 8, 2, 64, B, 64, L)
    one, two = (example.random_block(*args, page=16, fmt="mxfp8", seed=3) for _ in range(2))
    x = torch.randn(B * L, d, device=DEV).to(BF)
    want = []
    for _ in range(6):
        one.cache.seq_lens.add_(L)
        want.append([t.clone() for t in one.step(x, None, L)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):  # the attention's workspace is first asked for inside
            two.cache.seq_lens.add_(L)
            got = two.step(x, None, L)
        for w in want[:3]:
            graph.replay()
            side.synchronize()
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
        two.cache.seq_lens.add_(L)  # and a call outside the graph does not use the graph's
        out = two.step(x, None, L)
        side.synchronize()
        assert torch.equal(out[0], want[3][0]) and torch.equal(out[1], want[3][1])
        for w in want[4:]:
            graph.replay()
            side.synchronize()
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


def test_the_example_runs(example, capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["decode_block.py", "--requests", "2", "--context", "100", "--steps", "4"])
    example.main()
    assert "us a step" in capsys.readouterr().out
