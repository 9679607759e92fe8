"""The decode-step operators around the MoE layer (``include/moe_decode.h``): the residual addition with its
root-mean-square norm, and the paged key-value cache with the attention that reads it.

Like the rest of the binding these only check and marshal arguments; every step runs in the library's
kernels, asynchronously on the given stream (default: the current one).
"""
from __future__ import annotations

import ctypes

import torch

from . import MOE_ATTENTION_COUNTER_BYTES, MOE_OK, MoEError, _empty, _ok, _on_current_gpu, _on_stream, _raw_stream, lib, moe_attention_t, moe_kv_cache_t, moe_norm_t

MOE_KV_BF16, MOE_KV_MXFP8 = 0, 1
# The attention workspaces of calls outside captures, one for each GPU and stream, as large as the largest call so far: the
# calls of a stream run one after another, whatever their caches and shapes.
_WORKSPACES: dict[tuple[int, int], torch.Tensor] = {}

KV_STATUS = {1: "a sequence length outside the block table", 2: "a page index outside the cache"}


def _rows(t: torch.Tensor, name: str, shape, gpu: int, dtype=torch.bfloat16) -> tuple[int, int]:
    """Address and row stride of a row-strided 2-D tensor on cuda:gpu with contiguous columns."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != gpu:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on cuda:{gpu}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    row, col = t.stride()
    if col != 1 and shape[1] > 1:
        raise ValueError(f"the columns of {name} must be contiguous")
    if row == 0 and shape[0] > 1:  # the library reads stride 0 as contiguous rows
        raise ValueError(f"{name} is broadcast: its rows must lie in memory of their own")
    return t.data_ptr(), row


def moe_add_rms_norm(x: torch.Tensor, residual: torch.Tensor | None, weight: torch.Tensor, eps: float = 1e-6,
                     sum_out: torch.Tensor | None = None, y: torch.Tensor | None = None,
                     y_q: torch.Tensor | None = None, y_s: torch.Tensor | None = None, stream=None) -> None:
    """sum_out = bf16(x + residual); y = bf16((x + residual) * weight / rms); (y_q, y_s) = MXFP8(y).

    x, residual, sum_out, y: bf16 [T, d] (row-strided views allowed, broadcast rows not); weight: bf16 or fp32
    [d]; y_q: uint8 [T, d] E4M3 codes and y_s: uint8 [T, d / 32] E8M0 bytes, contiguous, as ``moe_permute``
    writes them.
    residual and each output may be None; sum_out may be x or residual, y may be x."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x must be [T, d], got {tuple(shape)}")
    T, d = shape
    gpu = x.get_device()
    if gpu < 0:
        raise ValueError(f"x must be a CUDA tensor, got one on {x.device}")
    _on_current_gpu("x", gpu)
    w32 = weight.dtype is torch.float32
    if not (w32 or weight.dtype is torch.bfloat16) or weight.shape != (d,) or not weight.is_contiguous() or \
            weight.get_device() != gpu:
        raise ValueError(f"weight must be a contiguous bf16 or fp32 tensor of {d} columns on cuda:{gpu}")
    xp, xs = _rows(x, "x", shape, gpu)
    rp, rs = (None, 0) if residual is None else _rows(residual, "residual", shape, gpu)
    up, us = (None, 0) if sum_out is None else _rows(sum_out, "sum_out", shape, gpu)
    yp, ys = (None, 0) if y is None else _rows(y, "y", shape, gpu)
    qp = sp = None
    if y_q is not None:
        qp, row = _rows(y_q, "y_q", shape, gpu, torch.uint8)
        if row != d and T > 1:
            raise ValueError("y_q must be contiguous")
    if y_s is not None:
        sp, row = _rows(y_s, "y_s", (T, d // 32), gpu, torch.uint8)
        if row != d // 32 and T > 1:
            raise ValueError("y_s must be contiguous")
    if T <= 1:  # the stride of a lone row means nothing
        xs = rs = us = ys = 0
    status = lib().moe_add_rms_norm(moe_norm_t(xp, rp, weight.data_ptr(), up, yp, qp, sp, xs, rs, us, ys, T, d, w32, eps),
                                    _raw_stream(stream))
    if status:
        _ok("moe_add_rms_norm", status)


class PagedKVCache:
    """One layer's paged key-value cache over the caller's tensors.

    k, v: [n_pages, page_size, n_kv_heads, head_dim], bf16, or uint8 E4M3 codes (MXFP8) with k_scales,
    v_scales uint8 [..., head_dim / 32]; any strides with contiguous columns, the same for k and v.
    block_table: int32 [n_seqs, max_pages], contiguous; seq_lens: int32 [n_seqs], the tokens of every request
    including the ones of the current step.  Their contents may change between calls (in place).

    ``append`` writes a step's new keys and values; ``attend`` is the attention of the step's new tokens."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None):
        mx = k_scales is not None
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must be alike: [n_pages, page_size, n_kv_heads, head_dim], columns contiguous")
        if k.dtype != (torch.uint8 if mx else torch.bfloat16) or v.dtype != k.dtype:
            raise ValueError("k and v must be bf16, or uint8 E4M3 codes with k_scales and v_scales")
        if mx != (v_scales is not None):
            raise ValueError("k_scales and v_scales go together")
        n_pages, page, heads, d = k.shape
        if mx:
            for s in (k_scales, v_scales):
                if s.dtype != torch.uint8 or s.shape != (n_pages, page, heads, d // 32) or s.stride(3) != 1:
                    raise ValueError("scales must be uint8 [n_pages, page_size, n_kv_heads, head_dim / 32]")
                if any(n > 1 and 32 * a != b for n, a, b in zip(s.shape[:3], s.stride(), k.stride())):
                    raise ValueError("the scales' strides must be those of k and v divided by 32")
        if block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
            raise ValueError("block_table must be a contiguous int32 [n_seqs, max_pages]")
        if seq_lens.dtype != torch.int32 or seq_lens.shape != block_table.shape[:1] or not seq_lens.is_contiguous():
            raise ValueError("seq_lens must be a contiguous int32 [n_seqs]")
        tensors = [t for t in (k, v, block_table, seq_lens, k_scales, v_scales) if t is not None]
        if len({t.device for t in tensors}) != 1 or not k.is_cuda:
            raise ValueError("the cache's tensors must be on one CUDA device")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.block_table, self.seq_lens = block_table, seq_lens
        self.device, self.n_seqs, self.n_kv_heads, self.head_dim = k.device, seq_lens.shape[0], heads, d
        self.status = torch.zeros(1, dtype=torch.int32, device=k.device)
        st = [s if n > 1 else 0 for n, s in zip(k.shape[:3], k.stride())]  # strides of lone entries mean nothing
        self._c = moe_kv_cache_t(k.data_ptr(), v.data_ptr(), k_scales.data_ptr() if mx else None,
                                 v_scales.data_ptr() if mx else None, block_table.data_ptr(), seq_lens.data_ptr(),
                                 self.status.data_ptr(), *st, MOE_KV_MXFP8 if mx else MOE_KV_BF16, n_pages, page,
                                 heads, d, self.n_seqs, block_table.shape[1])
        self._ref = ctypes.byref(self._c)
        self._workspace_bytes = {}
        self._index = k.get_device()

    @classmethod
    def allocate(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, fmt: str = "bf16") -> "PagedKVCache":
        """A cache with zeroed pages of its own on the block table's device; fmt: "bf16" or "mxfp8"."""
        if fmt not in ("bf16", "mxfp8"):
            raise ValueError(f"unknown cache format {fmt!r}")
        shape, dev = (n_pages, page_size, n_kv_heads, head_dim), block_table.device
        if fmt == "bf16":
            return cls(*(torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in "kv"), block_table, seq_lens)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=dev) for _ in "kv")
        ks, vs = (torch.zeros((*shape[:3], head_dim // 32), dtype=torch.uint8, device=dev) for _ in "kv")
        return cls(k, v, block_table, seq_lens, ks, vs)

    def _step_rows(self, t: torch.Tensor, name: str, heads: int | None = None, dtype=torch.bfloat16):
        """(L, heads, row stride) of [n_seqs, L, heads, head_dim] whose rows (b, l) lie at one stride."""
        shape = t.shape
        if len(shape) != 4 or t.dtype is not dtype or t.get_device() != self._index or shape[0] != self.n_seqs or \
                shape[3] != self.head_dim or (heads is not None and shape[2] != heads):
            raise ValueError(f"{name} must be {dtype} [{self.n_seqs}, L, {heads or 'heads'}, {self.head_dim}] on "
                             f"{self.device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
        B, L, h, d = shape
        sb, sl, sh, sd = t.stride()
        if sd != 1 or (h > 1 and sh != d) or (B > 1 and L > 1 and sb != L * sl):
            raise ValueError(f"{name}: heads must be contiguous and the rows (request, token) at one stride")
        row = sl if L > 1 else sb
        if row == 0 and B * L > 1:  # the library reads stride 0 as contiguous rows
            raise ValueError(f"{name} is broadcast: its rows must lie in memory of their own")
        return L, h, 0 if B * L <= 1 else row

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
        """Write the step's L new tokens: bf16 [n_seqs, L, n_kv_heads, head_dim], token l of request b at
        position seq_lens[b] - L + l (negative positions are skipped)."""
        _on_current_gpu("the cache", self._index)
        L, _, ks = self._step_rows(k_new, "k_new", self.n_kv_heads)
        Lv, _, vs = self._step_rows(v_new, "v_new", self.n_kv_heads)
        if L != Lv:
            raise ValueError("k_new and v_new hold different numbers of tokens")
        status = lib().moe_kv_append(self._ref, k_new.data_ptr(), ks, v_new.data_ptr(), vs, L, _raw_stream(stream))
        if status:
            _ok("moe_kv_append", status)

    def _bytes(self, n_q_heads: int, L: int) -> int:
        n = self._workspace_bytes.get((n_q_heads, L))
        if n is None:
            n = int(lib().moe_paged_attention_workspace(self._ref, n_q_heads, L))
            if n == 0:
                raise MoEError("moe_paged_attention_workspace", 1, lib().moe_last_error().decode())
            self._workspace_bytes[n_q_heads, L] = n
        return n

    def attention_workspace(self, n_q_heads: int, L: int, stream=None) -> torch.Tensor:
        """A workspace for ``attend`` of up to L new tokens, ready for calls on `stream`: for a program that captures its
        calls into graphs, or runs them on several streams.  It serves any calls that run one after another."""
        ws = _empty((self._bytes(n_q_heads, L),), torch.uint8, self.device, stream)
        with _on_stream(stream, self.device):
            ws[:MOE_ATTENTION_COUNTER_BYTES].zero_()
        return ws

    def _workspace(self, n_q_heads: int, L: int, stream, raw: int) -> torch.Tensor:
        if stream is None:
            capturing = torch._C._cuda_isCurrentStreamCapturing()
        else:
            with _on_stream(stream, self.device):
                capturing = torch._C._cuda_isCurrentStreamCapturing()
        if capturing:  # a graph may be replayed on any stream: it has a workspace of its own, cleared at every replay
            return self.attention_workspace(n_q_heads, L, stream)
        ws = _WORKSPACES.get((self._index, raw))
        if ws is None or ws.numel() < self._bytes(n_q_heads, L):
            _WORKSPACES[self._index, raw] = ws = self.attention_workspace(n_q_heads, L, stream)
        return ws

    def attend(self, q: torch.Tensor, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               scale: float | None = None, stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
        """Attention of the L newest tokens of every request: q, out bf16 [n_seqs, L, n_q_heads, head_dim]; lse
        fp32 [n_seqs, L, n_q_heads] or None; scale defaults to head_dim ** -0.5.  Row l sees the positions below
        seq_lens[b] - L + 1 + l; a row that sees nothing gives 0 (lse -inf).  An out that is not given is allocated on
        `stream`.

        workspace: one of ``attention_workspace`` (or uint8 memory whose first MOE_ATTENTION_COUNTER_BYTES bytes are
        zero); calls in it must not overlap, replays of graphs that captured them included.  Without it the calls of
        a stream share one of their own, and a captured call gets one that its graph clears before every run."""
        _on_current_gpu("the cache", self._index)
        L, heads, qs = self._step_rows(q, "q")
        if out is None:
            out = _empty(q.shape, q.dtype, self.device, stream)
        Lo, _, os_ = self._step_rows(out, "out", heads)
        if Lo != L:
            raise ValueError("q and out hold different numbers of tokens")
        if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:3] or not lse.is_contiguous() or
                                lse.get_device() != self._index):
            raise ValueError(f"lse must be a contiguous fp32 tensor of shape {tuple(q.shape[:3])}")
        if q.numel() == 0:
            return out
        raw = _raw_stream(stream)
        ws = self._workspace(heads, L, stream, raw) if workspace is None else workspace
        if workspace is not None and (ws.dtype != torch.uint8 or ws.get_device() != self._index or not ws.is_contiguous()):
            raise ValueError(f"workspace must be contiguous uint8 memory on {self.device}")
        a = moe_attention_t(q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), ws.data_ptr(),
                            ws.numel(), qs, os_, heads, L,
                            self.head_dim ** -0.5 if scale is None else scale)
        status = lib().moe_paged_attention(self._ref, ctypes.byref(a), raw)
        if status:
            _ok("moe_paged_attention", status)
        return out

    def check(self) -> None:
        """Wait for the device, then raise if a call met a bad length or page since the last check."""
        bits = int(self.status.item())
        if bits != MOE_OK:
            self.status.zero_()
            raise MoEError("PagedKVCache", 5, "; ".join(t for b, t in KV_STATUS.items() if bits & b))
