"""Argument checks of the decode-step calls: every refusal is made on the host, before any work, without a GPU."""
import ctypes

import pytest
import torch

P = 4096  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def m():
    import __graft_entry__ as g
    g.build_cuda()
    import block_scaled_fp4_sqrt_gb300 as mod
    return mod


def norm_args(m, **kw):
    a = dict(x=P, residual=P, weight=P, sum=P * 2, y=P * 3, y_q=P * 4, y_s=P * 5, x_stride=0, residual_stride=0,
             sum_stride=0, y_stride=0, T=2, d=64, weight_f32=0, eps=1e-6)
    a.update(kw)
    s = m.moe_norm_t()
    for k, v in a.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw", [dict(x=None), dict(weight=None), dict(sum=None, y=None, y_q=None, y_s=None),
                                dict(y_q=None), dict(y_s=None), dict(x=P + 2), dict(y=P + 8), dict(x_stride=63),
                                dict(x_stride=68), dict(sum_stride=8), dict(T=-1), dict(eps=-1.0),
                                dict(eps=float("nan"))])
def test_norm_refuses(m, kw):
    assert m.lib().moe_add_rms_norm(ctypes.byref(norm_args(m, **kw)), None) == 1
    assert b"moe_add_rms_norm" in m.lib().moe_last_error()


@pytest.mark.parametrize("kw", [dict(d=0), dict(d=60), dict(d=40), dict(d=65536 + 32)])
def test_norm_refuses_widths(m, kw):
    assert m.lib().moe_add_rms_norm(ctypes.byref(norm_args(m, **kw)), None) in (1, 2)


def test_norm_null_arguments(m):
    assert m.lib().moe_add_rms_norm(None, None) == 1


def cache(m, **kw):
    a = dict(k=P, v=P, k_s=P, v_s=P, block_table=P, seq_lens=P, status=P, page_stride=2048, row_stride=128,
             head_stride=128, format=m.MOE_KV_MXFP8 if hasattr(m, "MOE_KV_MXFP8") else 1, n_pages=4, page_size=16,
             n_kv_heads=1, head_dim=128, n_seqs=2, max_pages=2)
    a.update(kw)
    s = m.moe_kv_cache_t()
    for k, v in a.items():
        setattr(s, k, v)
    return s


BAD_CACHES = [dict(format=2), dict(format=-1), dict(head_dim=96), dict(head_dim=256), dict(page_size=0),
              dict(n_kv_heads=0), dict(n_pages=-1), dict(n_seqs=-1), dict(max_pages=-1), dict(max_pages=1 << 30),
              dict(n_seqs=(1 << 20) + 1), dict(row_stride=130), dict(page_stride=-32), dict(head_stride=8),
              dict(block_table=None), dict(seq_lens=None), dict(k=None), dict(v=None), dict(k_s=None), dict(v_s=None),
              dict(k=P + 8), dict(v=P + 1), dict(k_s=P + 2), dict(row_stride=32), dict(block_table=P + 2),
              dict(seq_lens=P + 1), dict(status=P + 3)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_caches_are_refused_by_every_call(m, kw):
    L = m.lib()
    c = cache(m, **kw)
    att = m.moe_attention_t(P, P, None, P, 1 << 30, 0, 0, 4, 1, 1.0)
    assert L.moe_kv_append(ctypes.byref(c), P, 0, P, 0, 1, None) in (1, 2)
    assert L.moe_last_error()
    assert L.moe_paged_attention(ctypes.byref(c), ctypes.byref(att), None) in (1, 2)
    assert L.moe_paged_attention_workspace(ctypes.byref(c), 4, 1) == 0


def test_append_refuses(m):
    L, c = m.lib(), cache(m)
    for args in ((None, 0, P, 0, 1), (P, 0, None, 0, 1), (P + 2, 0, P, 0, 1), (P, 0, P + 8, 0, 1), (P, 4, P, 0, 1),
                 (P, 0, P, 100, 1), (P, 0, P, 0, -1)):
        assert L.moe_kv_append(ctypes.byref(c), *args, None) == 1, args
    assert L.moe_kv_append(None, P, 0, P, 0, 1, None) == 1


def test_attention_refuses(m):
    L, c = m.lib(), cache(m, n_kv_heads=2, row_stride=256)
    n = L.moe_paged_attention_workspace(ctypes.byref(c), 4, 1) if torch.cuda.is_available() else 1 << 30
    good = dict(q=P, out=P, lse=None, workspace=P, workspace_bytes=n, q_stride=0, out_stride=0, n_q_heads=4, L=1,
                scale=1.0)
    for kw in (dict(q=None), dict(out=None), dict(workspace=None), dict(q=P + 2), dict(out=P + 8), dict(lse=P + 2),
               dict(workspace=P + 128), dict(q_stride=12), dict(out_stride=100), dict(n_q_heads=3), dict(n_q_heads=0),
               dict(L=-1), dict(scale=float("inf")), dict(scale=float("nan"))):
        a = m.moe_attention_t(*{**good, **kw}.values())
        # the workspace's size depends on the GPU: MOE_ERR_WORKSPACE there, MOE_ERR_CUDA without one
        want = (3 if torch.cuda.is_available() else 4) if "workspace" in kw else 1
        assert L.moe_paged_attention(ctypes.byref(c), ctypes.byref(a), None) == want, kw
    assert L.moe_paged_attention(None, ctypes.byref(m.moe_attention_t(*good.values())), None) == 1
    assert L.moe_paged_attention(ctypes.byref(c), None, None) == 1


def test_few_refuses_without_handles(m):
    assert m.lib().moe_forward_few(None, None, None, None, None, None, None, None, None) == 1


def test_python_calls_refuse_what_the_library_cannot_see(m):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    for bad in (lambda: m.moe_add_rms_norm(x, None, w, y=x),                      # not on a GPU
                lambda: m.moe_add_rms_norm(x[0], None, w),                        # not [T, d]
                lambda: m.moe_add_rms_norm(x, None, w[:32]),                      # another width
                lambda: m.moe_add_rms_norm(x, None, w.half())):                   # another type
        with pytest.raises(ValueError):
            bad()
    k = torch.zeros(4, 16, 1, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    scales = torch.zeros(4, 16, 1, 4, dtype=torch.uint8)
    u8 = k.to(torch.uint8)
    for args in ((k, k, table, lens), (k, k[:3], table, lens), (k, k.transpose(0, 1), table, lens),
                 (k, k, table.long(), lens), (k, k, table, lens[:1]), (k, k, table[:, ::2], lens),
                 (k, k, table, lens, scales, scales), (u8, u8, table, lens, scales),
                 (u8, u8, table, lens, scales[..., :2], scales[..., :2]), (u8, u8, table, lens)):
        with pytest.raises(ValueError):
            m.PagedKVCache(*args)
    with pytest.raises(ValueError):
        m.PagedKVCache.allocate(4, 16, 1, 128, table, lens, "fp4")
