"""A decoder block's step over a paged cache, with the library's operators in the order in which a server runs them:

  add + norm -> q, k, v projection -> cache append -> attention -> output projection -> add + norm -> MoE layer

With a rotation (``rope``) the queries and keys are normed a head, turned to their positions and appended in one call.

``DecoderBlock`` holds the block's weights, its cache and its MoE layer; ``step`` advances every request by L
tokens (1: decoding; more: a verify step's drafts).  The two dense projections are plain matrix products and stay
with torch; everything else is one library call each.  The MoE layer's output travels as the next block's ``x``
with the residual stream beside it, so that no addition has a kernel of its own.

Run it: ``python examples/decode_block.py --requests 4 --tokens 1 --steps 64`` prints the time of one block's step,
replayed from a CUDA graph, on random weights.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_sqrt_gb300 as moe  # noqa: E402

# The most rows for forward_few: its one kernel leads while launches and routing weigh most (one row of the full-size
# layer 34 us against 44), is near MoELayer.forward at three and four rows (67 and 82 against 64 and 81; ahead on smaller
# layers) and behind its tensor-memory GEMMs above.
FEW_ROWS = 4


class DecoderBlock:
    def __init__(self, layer: moe.MoELayer, cache: moe.PagedKVCache, n_q_heads: int, norm_attn, norm_moe, w_qkv, w_o,
                 eps: float = 1e-6, max_new: int = 1, rope: moe.RotaryPlan | None = None, q_norm=None, k_norm=None):
        """norm_*: [d]; w_qkv: bf16 [(n_q + 2 n_kv) head_dim, d]; w_o: bf16 [d, n_q head_dim].  max_new: the most new
        tokens of a step whose attention runs in the block's workspace (the blocks of a model may share one).  rope, q_norm,
        k_norm [head_dim]: the rotation and the heads' norms (None: without)."""
        self.layer, self.cache, self.n_q, self.eps = layer, cache, n_q_heads, eps
        self.norm_attn, self.norm_moe, self.w_qkv, self.w_o = norm_attn, norm_moe, w_qkv, w_o
        self.n_kv, self.hd, self.max_new = cache.n_kv_heads, cache.head_dim, max_new
        self.rope, self.q_norm, self.k_norm = rope, q_norm, k_norm
        self.workspace = cache.attention_workspace(n_q_heads, max_new)  # a captured step need not clear one

    def step(self, x: torch.Tensor, residual: torch.Tensor | None, L: int):
        """x: bf16 [n_seqs * L, d], the block before's MoE output (or the embedding), residual: the stream beside it
        (None at the first block).  The cache's ``seq_lens`` include the L new tokens.  Returns (x, residual)."""
        B, T = self.cache.n_seqs, x.shape[0]
        stream, y = torch.empty_like(x), torch.empty_like(x)
        moe.moe_add_rms_norm(x, residual, self.norm_attn, self.eps, sum_out=stream, y=y)
        qkv = (y @ self.w_qkv.t()).view(B, L, self.n_q + 2 * self.n_kv, self.hd)
        q, k, v = qkv.split((self.n_q, self.n_kv, self.n_kv), dim=2)  # views: the calls take the rows' stride
        if self.rope is None:
            self.cache.append(k, v)
        else:  # in place: q is a view of qkv
            self.cache.append_rotated(q, k, v, self.rope, None, self.q_norm, self.k_norm, self.eps, q_out=q)
        o = torch.empty((B, L, self.n_q, self.hd), dtype=x.dtype, device=x.device)
        self.cache.attend(q, out=o, workspace=self.workspace if L <= self.max_new else None)
        a = o.view(T, -1) @ self.w_o.t()
        moe.moe_add_rms_norm(a, stream, self.norm_moe, self.eps, sum_out=stream, y=y)
        return (self.layer.forward_few(y) if T <= FEW_ROWS else self.layer.forward(y)), stream


def random_block(d: int, f: int, E: int, k: int, n_q: int, n_kv: int, hd: int, n_seqs: int, max_len: int, L: int,
                 page: int = 64, fmt: str = "mxfp8", seed: int = 0, device="cuda:0", rotary: bool = False) -> DecoderBlock:
    """A block with random weights and an empty cache of its own pages; rotary: with head norms and a rotation."""
    g = torch.Generator(device=device).manual_seed(seed)

    def rand(*shape, std):
        return torch.empty(shape, dtype=torch.float32, device=device).normal_(0, std, generator=g)

    def codes(n, rows, cols):  # any E2M1 codes; scales near 1 / sqrt(cols)
        e = 127 - 2 - cols.bit_length() // 2
        return (torch.randint(0, 256, (n, rows, cols // 2), dtype=torch.uint8, device=device, generator=g),
                torch.randint(e - 1, e + 1, (n, rows, cols // 32), dtype=torch.uint8, device=device, generator=g))

    def experts(n):
        return moe.DeviceExperts(*codes(n, 2 * f, d), *codes(n, d, f))

    layer = moe.MoELayer(d, f, E, k, experts(E), experts(1), rand(E, d, std=d ** -0.5), rand(E, std=0.05),
                         max_T=n_seqs * L, device=device)
    pages = (max_len + page - 1) // page
    order = torch.randperm(n_seqs * pages, device=device, generator=g).to(torch.int32).view(n_seqs, pages)
    lens = torch.zeros(n_seqs, dtype=torch.int32, device=device)
    cache = moe.PagedKVCache.allocate(n_seqs * pages, page, n_kv, hd, order, lens, fmt)
    bf = torch.bfloat16
    rot = dict(rope=moe.RotaryPlan([10000.0 ** (-2 * i / hd) for i in range(hd // 2)], device=device),
               q_norm=(1 + rand(hd, std=0.1)).to(bf), k_norm=(1 + rand(hd, std=0.1)).to(bf)) if rotary else {}
    return DecoderBlock(layer, cache, n_q, (1 + rand(d, std=0.1)).to(bf), (1 + rand(d, std=0.1)).to(bf),
                        rand((n_q + 2 * n_kv) * hd, d, std=d ** -0.5).to(bf),
                        rand(d, n_q * hd, std=(n_q * hd) ** -0.5).to(bf), max_new=L, **rot)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=1, help="new tokens of every request in a step")
    ap.add_argument("--context", type=int, default=2000, help="tokens in the cache before the first step")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--cache", choices=("bf16", "mxfp8", "mxfp4"), default="mxfp8")
    ap.add_argument("--rotary", action="store_true", help="norms of the heads and a rotation before the cache")
    a = ap.parse_args()
    B, L, d = a.requests, a.tokens, 4096
    # three untimed steps run before the graph's
    block = random_block(d, 2048, 256, 6, 32, 4, 128, B, a.context + L * (a.steps + 3), L, fmt=a.cache, rotary=a.rotary)
    block.cache.seq_lens.fill_(a.context)
    x0 = torch.randn(B * L, d, device="cuda:0").to(torch.bfloat16)

    def step():
        block.cache.seq_lens.add_(L)
        return block.step(x0, None, L)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())  # where the weights, lengths and x0 are still being written
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        e0.record()
        for _ in range(a.steps):
            graph.replay()
        e1.record()
        side.synchronize()
    block.cache.check()
    block.layer.check()
    print(f"{B} requests x {L} tokens, {a.context} cached, {a.cache} cache: "
          f"{1e3 * e0.elapsed_time(e1) / a.steps:.1f} us a step")


if __name__ == "__main__":
    main()
