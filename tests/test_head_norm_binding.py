"""Calls of the head norms' binding that its documentation allows, against a library that only records them."""
import itertools

import pytest
import torch

from test_cache_ops_abi import b, plan  # noqa: F401
from test_decode_binding import OnGpu, m as traced, zeros  # noqa: F401

I32 = torch.int32


@pytest.mark.parametrize("lead", [(0,), (0, 2), (2, 0), (3, 2, 0), (3, 0, 2), (0, 0), (1, 0, 1), (2, 0, 3, 2)])
def test_no_rows_in_any_shape(b, lead):  # noqa: F811
    n = len(b.library.calls)
    q, k = zeros(*lead, 8, 64), zeros(*lead, 2, 64)
    out = b.moe_head_norm_rope(q, k, plan(b), zeros(1, 0, dtype=I32), zeros(64), zeros(64), q_out=zeros(*lead, 8, 64), k_out=k)
    a = b.library.calls[-1][1][1]
    assert len(b.library.calls) == n + 1 and (a.T, a.n_q_heads, a.n_kv_heads, a.head_dim) == (0, 8, 2, 64)
    assert out[0].shape == q.shape and out[1] is k


def test_no_rows_of_heads_that_lie_apart(b):  # noqa: F811
    calls = len(b.library.calls)
    q = OnGpu(torch.zeros(2, 0, 64, 8, dtype=torch.bfloat16).transpose(2, 3))
    with pytest.raises(ValueError, match="contiguous"):
        b.moe_head_norm_rope(q, None, plan(b), zeros(1, 0, dtype=I32), q_out=zeros(2, 0, 8, 64))
    assert len(b.library.calls) == calls


def test_rows_in_any_shape(b):  # noqa: F811
    for lead in itertools.chain(itertools.product((1, 2, 3), repeat=3), itertools.product((1, 4), repeat=2)):
        rows = 1
        for x in lead:
            rows *= x
        b.moe_head_norm_rope(zeros(*lead, 8, 64), None, plan(b), zeros(1, rows, dtype=I32), q_out=zeros(*lead, 8, 64))
        a = b.library.calls[-1][1][1]
        assert a.T == rows and a.q_stride == (512 if rows > 1 else 0)
