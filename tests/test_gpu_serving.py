"""The operators around the paged cache run together as a server runs them: pages are taken, copied and given back, queries and
keys normed, turned and appended, and the attention reads them; and the decoder block of the example with all of it."""
import os
import sys

import pytest
import torch

import test_gpu_cache_fp4 as fp4
import test_gpu_decode as dec
from test_gpu_decode import BF, DEV, gen, moe, randn  # noqa: F401
from test_gpu_rope import freqs, reference as turned

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("D,kv,group,page", [(64, 2, 4, 16), (128, 1, 8, 5)])
def test_verify_steps_with_branches_and_rejected_drafts(moe, fmt, D, kv, group, page):  # noqa: F811
    """Requests grow by drafts of which some are rejected, branch, end and begin again; every step's attention against 64 bits
    over what the cache should hold (the tokens' own rows, kept beside it)."""
    n_seqs, n_pages, max_pages, rot, L = 5, 120, 24, D // 2, 4
    g = gen(D + page)
    pool = moe.PagePool.allocate(n_seqs, max_pages, n_pages, page, DEV)
    cache = moe.PagedKVCache.allocate(n_pages, page, kv, D, pool.block_table, pool.seq_lens, fmt)
    plan = moe.RotaryPlan(freqs(rot), device=DEV)
    qw, kw = ((1 + 0.2 * randn(g, D)).to(BF) for _ in "qk")
    copies = torch.empty(n_seqs, 2, dtype=torch.int32, device=DEV)
    held = [0] * n_seqs  # the model's lengths
    tokens = [[] for _ in range(n_seqs)]  # (k, v) rows before the norm, by position

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def step(grow, L):
        """Requests with grow[b] take L tokens, the others none (they take part as empty rows behind the last)."""
        new = [n + (L if x else 0) for n, x in zip(held, grow)]
        pool.resize(i32(new), copies)
        moe.moe_copy_pages([cache], copies)
        qkv = randn(g, n_seqs, L, (group + 2) * kv, D).to(BF)
        q, k, v = qkv.split((group * kv, kv, kv), dim=2)
        q_raw = q.clone()
        lens = [n if x else 0 for n, x in zip(new, grow)]  # what this step sees of a request
        saved = pool.seq_lens.clone()
        pool.seq_lens.copy_(i32(lens))
        out_q = cache.append_rotated(q, k, v, plan, None, qw, kw)
        out = cache.attend(out_q)
        for b in range(n_seqs):
            if not grow[b]:
                assert torch.all(out[b] == 0)
                continue
            tokens[b] += [(k[b, l].clone(), v[b, l].clone()) for l in range(L)]
            pos = torch.arange(new[b] - L, new[b], device=DEV)[None]
            ref, bound = turned(q_raw[b], qw, 1e-6, pos, freqs(rot), None, "half")
            assert torch.all((out_q[b].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1.01 * bound + 1e-38)
        check = fp4.check_attend if fmt == "mxfp4" else dec.check_attend
        cache.tab = pool.block_table.cpu()
        check(cache, out_q, lens)
        # and what the cache holds is what its tokens were
        for b in range(n_seqs):
            if grow[b]:
                n = new[b]
                ks, vs = (torch.stack([t[i] for t in tokens[b]]) for i in (0, 1))
                want, _ = turned(ks, kw, 1e-6, torch.arange(n, device=DEV)[None], freqs(rot), None, "half")
                rows = fp4.rows_of if fmt == "mxfp4" else dec.rows_of
                # Of a block's largest element: half a step of bf16 and the norm's fp32; MX blocks scale it into
                # [2^8, 2^9) or [4, 8), where 512 would become 448 and 8 would become 6, more than any rounding is off by.
                tol = {"bf16": 2.0 ** -8 * 1.01, "mxfp8": 0.126, "mxfp4": 0.251}[fmt]
                for got, ref in ((rows(cache, b, n, "k"), want), (rows(cache, b, n, "v"), vs.double())):
                    top = ref.abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)
                    assert torch.all((got - ref).abs() <= tol * top)
        pool.seq_lens.copy_(saved)
        held[:] = new
        pool.check()
        cache.check()

    step([True, True, False, False, True], 21)
    step([True, False, False, False, True], L)
    pool.resize(i32([held[0] - 2, held[1], 0, 0, held[4]]), copies)  # two drafts of the first are rejected
    held[0] -= 2
    del tokens[0][held[0]:]
    pool.fork(i32([0, 1]), i32([2, 3]))
    held[2], held[3] = held[0], held[1]
    tokens[2], tokens[3] = list(tokens[0]), list(tokens[1])
    step([True, True, True, True, True], L)
    pool.resize(i32([0, held[1], held[2], held[3], 0]), copies)  # two requests end
    for b in (0, 4):
        held[b], tokens[b] = 0, []
    moves = pool.compact(torch.empty(n_pages // 2, 2, dtype=torch.int32, device=DEV))
    moe.moe_copy_pages([cache], moves)
    live = int((pool.page_refs > 0).sum())
    assert torch.all(pool.page_refs[:live] > 0) and torch.all(pool.page_refs[live:] == 0)
    step([True, True, True, True, False], L)
    step([True, False, False, True, True], 1)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("rotary", [False, True])
def test_the_example_block_runs_with_every_cache(moe, fmt, rotary):  # noqa: F811
    """The block's step, eagerly and replayed from a graph: the same bits; its attention half against 64 bits is tested above."""
    from decode_block import random_block
    B, L, d = 3, 2, 256
    outs = []
    for replay in (False, True):
        block = random_block(d, 128, 8, 2, 8, 2, 64, B, 64, L, page=16, fmt=fmt, seed=3, rotary=rotary)
        g = gen(9)
        x = randn(g, B * L, d).to(BF)
        block.cache.seq_lens.fill_(L)
        if replay:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                block.step(x, None, L)
                side.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    y, stream = block.step(x, None, L)
                for _ in range(3):
                    graph.replay()
                    block.cache.seq_lens.add_(L)
            side.synchronize()
        else:
            for _ in range(3):
                y, stream = block.step(x, None, L)
                block.cache.seq_lens.add_(L)
        torch.cuda.synchronize()
        block.cache.check()
        block.layer.check()
        outs.append((y.clone(), stream.clone()))
    for a, b in zip(*outs):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_the_example_prints_a_step(moe, monkeypatch, capsys):  # noqa: F811
    import decode_block
    monkeypatch.setattr(sys, "argv", ["decode_block.py", "--requests", "2", "--steps", "3", "--context", "100", "--cache", "mxfp4",
                                      "--rotary"])
    decode_block.main()
    assert "mxfp4 cache" in capsys.readouterr().out
