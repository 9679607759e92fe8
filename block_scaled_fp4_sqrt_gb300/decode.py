"""The decode-step operators around the MoE layer (``include/moe_decode.h``): the residual addition with its
root-mean-square norm, the norms of the heads with the position rotation, the paged key-value cache with the attention
that reads it, and the pool of its pages.

Like the rest of the binding these only check and marshal arguments; every step runs in the library's
kernels, asynchronously on the given stream (default: the current one).
"""
from __future__ import annotations

import ctypes
from fractions import Fraction

import torch

from . import (MOE_ATTENTION_COUNTER_BYTES, MOE_OK, MoEError, _empty, _ok, _on_current_gpu, _on_stream, _raw_stream,
               _refuse, lib, moe_attention_t, moe_head_rope_t, moe_kv_cache_t, moe_norm_t, moe_page_pool_t)

MOE_KV_BF16, MOE_KV_MXFP8, MOE_KV_MXFP4 = 0, 1, 4
# The attention workspaces of calls outside captures, one for each GPU and stream, as large as the largest call so far: the
# calls of a stream run one after another, whatever their caches and shapes.
_WORKSPACES: dict[tuple[int, int], torch.Tensor] = {}

KV_STATUS = {1: "a sequence length outside the block table", 2: "a page index outside the cache",
             4: "a request wanted more pages than are free", 8: "a fork between requests that do not allow it"}
MOE_POOL_MAX_SEQS = 8192
PAIRS = {"half": 0, "adjacent": 1}
_CacheAt = ctypes.POINTER(moe_kv_cache_t)


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


# 2 pi to 40 digits: a frequency becomes a fraction of a turn without losing a bit of its 64
_TWO_PI = Fraction(6283185307179586476925286766559005768394, 10 ** 39)


class RotaryPlan:
    """The rotation of a model's heads: inv_freq [rot_dim / 2], the angle per position of every pair in radians (numbers or a
    tensor, read as 64-bit); pairs "half" (columns i and i + rot_dim / 2) or "adjacent" (2 i and 2 i + 1); axis_of
    [rot_dim / 2], the position axis that a pair turns with (None: one axis).  Kept as exact fractions of a turn, so that
    far positions lose nothing."""

    def __init__(self, inv_freq, axis_of=None, pairs: str = "half", device="cuda"):
        if pairs not in PAIRS:
            raise ValueError(f"unknown pairs {pairs!r}")
        freq = [float(f) for f in inv_freq]
        axis = None if axis_of is None else [int(a) for a in axis_of]
        if any(f != f or abs(f) == float("inf") for f in freq):
            raise ValueError("inv_freq must be finite")
        if axis is not None and (len(axis) != len(freq) or any(not 0 <= a < 256 for a in axis)):
            raise ValueError(f"axis_of must hold {len(freq)} axes in [0, 256)")
        turns = [round(Fraction(f) / _TWO_PI * 2 ** 64) % 2 ** 64 for f in freq]
        self.rot_dim, self.n_axes = 2 * len(freq), 1 + max(axis or [0])
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)
        self.axis = None if axis is None else torch.tensor(axis, dtype=torch.uint8, device=device)
        self.pairs = PAIRS[pairs]
        self.at, self.axis_at = self.turns.data_ptr() if freq else None, None if axis is None or not axis else self.axis.data_ptr()


def _head_rows(t: torch.Tensor, name: str, gpu: int) -> tuple:
    """(rows, heads, head_dim, row stride) of a bf16 tensor [..., heads, head_dim] whose rows lie at one stride."""
    shape = t.shape
    if len(shape) < 3 or t.dtype is not torch.bfloat16 or t.get_device() != gpu:
        raise ValueError(f"{name} must be bf16 [..., heads, head_dim] on cuda:{gpu}, got {t.dtype} {tuple(shape)} on {t.device}")
    *lead, h, d = shape
    *steps, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"{name}: heads must be contiguous")
    if 0 in lead:  # no rows: their strides mean nothing
        return 0, h, d, 0
    rows, row = 1, 0
    for n, s in zip(reversed(lead), reversed(steps)):
        if n != 1:
            if rows == 1:
                row = s
                if row == 0:  # the library reads stride 0 as contiguous rows
                    raise ValueError(f"{name} is broadcast: its rows must lie in memory of their own")
            elif s != rows * row:
                raise ValueError(f"{name}: the rows must lie at one stride")
            rows *= n
    return rows, h, d, row


def _head_weights(q_weight, k_weight, dim: int, gpu: int) -> tuple:
    """Addresses of the two weights (None: no norm) and whether they are fp32."""
    at, kind = [], None
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is None:
            at.append(None)
            continue
        dtype = w.dtype
        if (dtype is not torch.bfloat16 and dtype is not torch.float32) or (kind is not None and dtype is not kind) or \
                w.shape != (dim,) or not w.is_contiguous() or w.get_device() != gpu:
            raise ValueError(f"{name} must be a contiguous bf16 or fp32 tensor of {dim} columns on cuda:{gpu}, of the other "
                             "weight's type")
        kind = dtype
        at.append(w.data_ptr())
    return at[0], at[1], kind is torch.float32


def _head_positions(positions, rope: "RotaryPlan", rows: int, gpu: int):
    if rope.turns.get_device() != gpu:
        raise ValueError(f"the rotation's plan lies on {rope.turns.device}, the tensors on cuda:{gpu}")
    if positions is None:
        return None
    if positions.dtype is not torch.int32 or positions.numel() != rope.n_axes * rows or not positions.is_contiguous() or \
            positions.get_device() != gpu:
        _refuse(positions, "positions", f"int32 [{rope.n_axes}, {rows}]")
    return positions.data_ptr()


def moe_head_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, rope: RotaryPlan, positions: torch.Tensor,
                       q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                       q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None) -> tuple:
    """Root-mean-square norm of every head of q and k and its rotation, in one pass; returns (q_out, k_out).

    q, k: bf16 [..., heads, head_dim] with the same rows, or None (views of a fused projection serve); positions: int32
    [n_axes, rows] contiguous (in any shape of that order); weights: [head_dim] bf16 or fp32, None for no norm.  q_out may be
    q and k_out k; outputs that are not given are allocated on `stream`."""
    lead = q if q is not None else k
    if lead is None:
        raise ValueError("q or k must be given")
    gpu = lead.get_device()
    if gpu < 0:
        raise ValueError(f"q and k must be CUDA tensors, got one on {lead.device}")
    _on_current_gpu("q" if q is not None else "k", gpu)
    rows, heads, dim, at = -1, [0, 0], -1, []
    for i, (name, t, out) in enumerate((("q", q, q_out), ("k", k, k_out))):
        if t is None:
            if out is not None:
                raise ValueError(f"{name}_out is given without {name}")
            at.append((None, None, 0, 0))
            continue
        n, h, d, step = _head_rows(t, name, gpu)
        if out is None:
            out = _empty(t.shape, t.dtype, t.device, stream)
        no, ho, do, step_out = _head_rows(out, name + "_out", gpu)
        if (no, ho, do) != (n, h, d) or (rows >= 0 and (rows, dim) != (n, d)):
            raise ValueError(f"{name} holds {n} rows of {h} heads of {d} columns, {name}_out {no} of {ho} of {do}, and q {rows} of "
                             f"heads of {dim}")
        rows, dim, heads[i] = n, d, h
        at.append((t.data_ptr(), out.data_ptr(), step, step_out))
        if i == 0:
            q_out = out
        else:
            k_out = out
    pos = _head_positions(positions, rope, rows, gpu)
    if pos is None and rows and rope.rot_dim:
        raise ValueError("positions must be given")
    qw, kw, w32 = _head_weights(q_weight, k_weight, dim, gpu)
    (qp, qop, qs, qos), (kp, kop, ks, kos) = at
    status = lib().moe_head_norm_rope(None, moe_head_rope_t(
        qp, kp, None, qop, kop, qw, kw, rope.at, rope.axis_at, pos, qs, ks, 0, qos, kos, 0, rows, 0, heads[0], heads[1], dim,
        rope.rot_dim, rope.pairs, rope.n_axes, w32, eps), _raw_stream(stream))
    if status:
        _ok("moe_head_norm_rope", status)
    return q_out, k_out


class PagedKVCache:
    """One layer's paged key-value cache over the caller's tensors.

    k, v: [n_pages, page_size, n_kv_heads, head_dim], bf16, or uint8 E4M3 codes (MXFP8) with k_scales,
    v_scales uint8 [..., head_dim / 32]; or uint8 [..., head_dim / 2] of two E2M1 codes each, the even column in the low
    half (MXFP4), with the same scales; any strides with contiguous columns, the same for k and v.
    block_table: int32 [n_seqs, max_pages], contiguous; seq_lens: int32 [n_seqs], the tokens of every request
    including the ones of the current step.  Their contents may change between calls (in place).

    ``append`` writes a step's new keys and values; ``attend`` is the attention of the step's new tokens."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None):
        mx = k_scales is not None
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must be alike: [n_pages, page_size, n_kv_heads, head_dim], columns contiguous")
        if k.dtype != (torch.uint8 if mx else torch.bfloat16) or v.dtype != k.dtype:
            raise ValueError("k and v must be bf16, or uint8 E4M3 or E2M1 codes with k_scales and v_scales")
        if mx != (v_scales is not None):
            raise ValueError("k_scales and v_scales go together")
        n_pages, page, heads, d = k.shape
        # codes of head_dim columns with head_dim / 32 scales: a byte a column, or half a byte
        per_byte = 2 if mx and k_scales.dim() == 4 and 16 * k_scales.shape[3] == d else 1
        d *= per_byte
        if mx:
            for s in (k_scales, v_scales):
                if s.dtype != torch.uint8 or s.shape != (n_pages, page, heads, d // 32) or s.stride(3) != 1:
                    raise ValueError("scales must be uint8 [n_pages, page_size, n_kv_heads, head_dim / 32]")
                if any(n > 1 and 32 * a != per_byte * b for n, a, b in zip(s.shape[:3], s.stride(), k.stride())):
                    raise ValueError("the scales' strides must be those of k and v, counted in columns, divided by 32")
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
        self.format = (MOE_KV_MXFP4 if per_byte == 2 else MOE_KV_MXFP8) if mx else MOE_KV_BF16
        st = [s * per_byte if n > 1 else 0 for n, s in zip(k.shape[:3], k.stride())]  # strides of lone entries mean nothing
        self._c = moe_kv_cache_t(k.data_ptr(), v.data_ptr(), k_scales.data_ptr() if mx else None,
                                 v_scales.data_ptr() if mx else None, block_table.data_ptr(), seq_lens.data_ptr(),
                                 self.status.data_ptr(), *st, self.format, n_pages, page,
                                 heads, d, self.n_seqs, block_table.shape[1])
        self._ref, self._at = ctypes.byref(self._c), ctypes.pointer(self._c)
        self._workspace_bytes = {}
        self._index = k.get_device()

    @classmethod
    def allocate(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, fmt: str = "bf16") -> "PagedKVCache":
        """A cache with zeroed pages of its own on the block table's device; fmt: "bf16", "mxfp8" or "mxfp4"."""
        if fmt not in ("bf16", "mxfp8", "mxfp4"):
            raise ValueError(f"unknown cache format {fmt!r}")
        shape, dev = (n_pages, page_size, n_kv_heads, head_dim), block_table.device
        if fmt == "bf16":
            return cls(*(torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in "kv"), block_table, seq_lens)
        codes = (*shape[:3], head_dim // 2) if fmt == "mxfp4" else shape
        k, v = (torch.zeros(codes, dtype=torch.uint8, device=dev) for _ in "kv")
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

    def append_rotated(self, q: torch.Tensor | None, k_new: torch.Tensor, v_new: torch.Tensor, rope: RotaryPlan,
                       positions: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                       k_weight: torch.Tensor | None = None, eps: float = 1e-6, q_out: torch.Tensor | None = None,
                       k_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
        """``moe_head_norm_rope`` of the step's L new tokens and ``append`` of the rotated keys and of the values, in one
        pass: q [n_seqs, L, n_q_heads, head_dim] or None, k_new, v_new [n_seqs, L, n_kv_heads, head_dim]; positions None:
        the tokens' places in their sequences.  Returns q_out (allocated on `stream` if not given; may be q); k_out, if given,
        receives the rotated keys as well."""
        _on_current_gpu("the cache", self._index)
        L, _, ks = self._step_rows(k_new, "k_new", self.n_kv_heads)
        Lv, _, vs = self._step_rows(v_new, "v_new", self.n_kv_heads)
        if L != Lv:
            raise ValueError("k_new and v_new hold different numbers of tokens")
        qp = qop = kop = None
        heads = qs = qos = kos = 0
        if q is not None:
            Lq, heads, qs = self._step_rows(q, "q")
            if q_out is None:
                q_out = _empty(q.shape, q.dtype, self.device, stream)
            Lo, _, qos = self._step_rows(q_out, "q_out", heads)
            if Lq != L or Lo != L:
                raise ValueError("q, q_out and k_new hold different numbers of tokens")
            qp, qop = q.data_ptr(), q_out.data_ptr()
        elif q_out is not None:
            raise ValueError("q_out is given without q")
        if k_out is not None:
            Lo, _, kos = self._step_rows(k_out, "k_out", self.n_kv_heads)
            if Lo != L:
                raise ValueError("k_out and k_new hold different numbers of tokens")
            kop = k_out.data_ptr()
        pos = _head_positions(positions, rope, self.n_seqs * L, self._index)
        qw, kw, w32 = _head_weights(q_weight, k_weight, self.head_dim, self._index)
        status = lib().moe_head_norm_rope(self._ref, moe_head_rope_t(
            qp, k_new.data_ptr(), v_new.data_ptr(), qop, kop, qw, kw, rope.at, rope.axis_at, pos, qs, ks, vs, qos, kos, 0, 0, L,
            heads, self.n_kv_heads, self.head_dim, rope.rot_dim, rope.pairs, rope.n_axes, w32, eps), _raw_stream(stream))
        if status:
            _ok("moe_head_norm_rope", status)
        return q_out

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
        _check_status(self.status, "PagedKVCache")


def _check_status(status: torch.Tensor, name: str) -> None:
    bits = int(status.item())
    if bits != MOE_OK:
        status.zero_()
        raise MoEError(name, 5, "; ".join(t for b, t in KV_STATUS.items() if bits & b))


class PagePool:
    """The pages of caches that share one block table, managed on the device without a host synchronisation.

    block_table int32 [n_seqs, max_pages], seq_lens int32 [n_seqs] (those of the caches) and page_refs int32 [n_pages], the
    number of requests that hold each page: contiguous, changed in place.  ``resize`` grows, truncates and frees, ``fork``
    branches, ``compact`` moves pages together; ``moe_copy_pages`` then copies the contents that they ask for, in every
    layer's cache, before the next append."""

    def __init__(self, block_table: torch.Tensor, seq_lens: torch.Tensor, page_refs: torch.Tensor, page_size: int):
        for name, t, dims in (("block_table", block_table, 2), ("seq_lens", seq_lens, 1), ("page_refs", page_refs, 1)):
            if t.dtype is not torch.int32 or t.dim() != dims or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of {dims} dimensions")
        if seq_lens.shape[0] != block_table.shape[0]:
            raise ValueError("seq_lens and block_table hold different numbers of requests")
        if len({t.device for t in (block_table, seq_lens, page_refs)}) != 1:
            raise ValueError("the pool's tensors must be on one CUDA device")
        if seq_lens.shape[0] > MOE_POOL_MAX_SEQS:
            raise ValueError(f"a pool holds up to {MOE_POOL_MAX_SEQS} requests")
        self.block_table, self.seq_lens, self.page_refs, self.page_size = block_table, seq_lens, page_refs, page_size
        self.device, self._index = block_table.device, block_table.get_device()
        self.n_seqs, self.max_pages, self.n_pages = *block_table.shape, page_refs.shape[0]
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._c = moe_page_pool_t(block_table.data_ptr(), seq_lens.data_ptr(), page_refs.data_ptr(), self.status.data_ptr(),
                                  self.n_seqs, self.max_pages, self.n_pages, page_size)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def allocate(cls, n_seqs: int, max_pages: int, n_pages: int, page_size: int, device="cuda") -> "PagePool":
        """A pool of its own tensors: every request empty, every page free."""
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.full((n_seqs, max_pages), -1, **i32), torch.zeros(n_seqs, **i32), torch.zeros(n_pages, **i32), page_size)

    def _ints(self, t: torch.Tensor, name: str, shape: tuple) -> int:
        if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous() or t.get_device() != self._index:
            _refuse(t, name, f"int32 {list(shape)} on {self.device}")
        return t.data_ptr()

    def fork(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Request dst[i], of length 0, becomes a branch of request src[i]: the same pages and length.  int32 [n]."""
        _on_current_gpu("the pool", self._index)
        n = src.shape[0] if src.dim() == 1 else -1
        status = lib().moe_pages_fork(self._ref, self._ints(src, "src", (n,)), self._ints(dst, "dst", (n,)), n, _raw_stream(stream))
        if status:
            _ok("moe_pages_fork", status)

    def resize(self, new_lens: torch.Tensor, copies: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Every request gets length new_lens[b] (int32 [n_seqs]): pages behind it go back, missing ones are taken.  Returns
        copies, int32 [n_seqs, 2] (allocated on `stream` if not given): (old page, new page) of the requests that grow inside a
        page that others hold too, for ``moe_copy_pages``, and (-1, -1).  A request whose pages are not to be had keeps its
        length (``check`` reports it)."""
        _on_current_gpu("the pool", self._index)
        if copies is None:
            copies = _empty((self.n_seqs, 2), torch.int32, self.device, stream)
        status = lib().moe_pages_resize(self._ref, self._ints(new_lens, "new_lens", (self.n_seqs,)),
                                        self._ints(copies, "copies", (self.n_seqs, 2)), _raw_stream(stream))
        if status:
            _ok("moe_pages_resize", status)
        return copies

    def compact(self, copies: torch.Tensor, stream=None) -> torch.Tensor:
        """Move the highest live pages into the lowest free ones, at most copies.shape[0] of them; copies, int32
        [capacity, 2], receives (from, to) of the moves for ``moe_copy_pages``, and (-1, -1)."""
        _on_current_gpu("the pool", self._index)
        n = copies.shape[0]
        status = lib().moe_pages_compact(self._ref, self._ints(copies, "copies", (n, 2)), n, _raw_stream(stream))
        if status:
            _ok("moe_pages_compact", status)
        return copies

    def free_pages(self) -> int:
        """The number of free pages (waits for the device)."""
        return int((self.page_refs == 0).sum())

    def check(self) -> None:
        """Wait for the device, then raise if a call met a bad table, or could not do what was asked, since the last check."""
        _check_status(self.status, "PagePool")


def moe_copy_pages(caches, copies: torch.Tensor, stream=None) -> None:
    """In every cache of the list, page copies[i, 1] receives the contents of page copies[i, 0]; pairs whose first page is
    negative are skipped.  copies: int32 [n, 2].  No page may be the second of two pairs, or of one and the first of another."""
    shape, gpu = copies.shape, copies.get_device()
    if len(shape) != 2 or shape[1] != 2 or copies.dtype is not torch.int32 or gpu < 0 or not copies.is_contiguous():
        _refuse(copies, "copies", "int32 [n, 2]")
    _on_current_gpu("copies", gpu)
    at = []
    for c in caches:
        if c._index != gpu:
            raise ValueError(f"a cache lies on {c.device}, copies on {copies.device}")
        at.append(c._at)
    if not at:
        return
    status = lib().moe_copy_pages((_CacheAt * len(at))(*at), len(at), copies.data_ptr(), shape[0], _raw_stream(stream))
    if status:
        _ok("moe_copy_pages", status)
