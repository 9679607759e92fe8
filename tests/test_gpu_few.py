"""moe_forward_few, the whole layer for up to eight tokens in one kernel, against the 64-bit oracle."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_support import (MEDIUM, TOL_WEIGHT_REL, WIDE, WORKLOADS, assert_close, bf16_to_f64, case, device, x_to_device)

pytestmark = pytest.mark.gpu


def run_few(layer, x, **kw):
    T, k = x.shape[0], layer.k
    ids = torch.full((T, k), -9, dtype=torch.int32, device=device())
    w = torch.full((T, k), -9.0, device=device())
    out = layer.forward_few(x, topk_ids=ids, topk_w=w, **kw)
    torch.cuda.synchronize()
    layer.check()
    return out, ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def check(name, T, seed=0):
    wl, inp, ids_ref, wts_ref, layer = case(name, T, seed)
    x = x_to_device(inp.x)
    out, ids, w = run_few(layer, x)
    assert np.array_equal(ids, ids_ref)
    assert np.max(np.abs(w - wts_ref) / np.abs(wts_ref)) <= TOL_WEIGHT_REL
    y_ref = oracle.layer(inp.x, ids_ref, wts_ref, inp.experts, inp.shared, wl.swiglu_limit)
    assert_close(bf16_to_f64(out), y_ref, f"{name} T={T}")
    assert np.array_equal(layer.last_topk_ids().cpu().numpy(), ids_ref)
    return wl, inp, layer, x, out


@pytest.mark.parametrize("T", [1, 2, 3, 5, 8])
def test_tiny(T):
    check("tiny", T)


@pytest.mark.parametrize("name,T", [("medium", 1), ("medium", 8), ("wide", 7), ("verify512", 1), ("verify512", 8),
                                    ("hash512", 5)])
def test_larger_layers(name, T):
    """Several items a block and several K groups an item; 384 experts (two selection widths); the full-size layer."""
    wl, inp, layer, x, out = check(name, T)
    again, _, _ = run_few(layer, x)  # the counters were left ready, and no order of arrival shows in the result
    assert torch.equal(again, out)


@pytest.mark.parametrize("d,f,E,k,T", [(256, 128, 1, 1, 8), (256, 128, 3, 3, 8), (512, 384, 5, 2, 4), (768, 640, 9, 4, 6),
                                       (8192, 128, 4, 2, 8), (4352, 256, 20, 16, 8)])
def test_odd_shapes(d, f, E, k, T):
    """Expert counts that several tokens share, K groups that do not fill the four splits, d beyond one pass."""
    wl = dataclasses.replace(MEDIUM, name=f"d{d}f{f}E{E}k{k}", T=T, d=d, f=f, E=E, k=k)
    WORKLOADS[wl.name] = wl
    check(wl.name, T)


def test_without_shared_expert_and_with_router_weights_per_call_or_resident():
    from block_scaled_fp4_sqrt_gb300 import MoELayer
    wl = MEDIUM.with_T(6)
    inp, ids_ref, wts_ref, _ = oracle.margin_filtered_layer(wl, 3)
    y_ref = oracle.layer(inp.x, ids_ref, wts_ref, inp.experts, None, wl.swiglu_limit)
    x = x_to_device(inp.x)
    outs = []
    for resident in (False, True):
        layer = MoELayer.from_host(inp, device=device(), max_T=6, with_shared=False, resident_router=resident)
        out, ids, _ = run_few(layer, x)
        assert np.array_equal(ids, ids_ref)
        assert_close(bf16_to_f64(out), y_ref, "no shared expert")
        outs.append(out)
    assert torch.equal(*outs)


def test_input_magnitudes():
    """x far from 1, blocks of very different size inside a token, zero tokens, clamped SwiGLU."""
    wl, inp, ids, wts, layer = case("tiny", 8)
    rng = np.random.default_rng(5)
    x = rng.standard_normal((8, wl.d)).astype(np.float32)
    x[0] = 0
    x[1] *= 30
    x[2] *= 2.0 ** -100
    x[3, :64] *= 2.0 ** -12
    x[4, 32:] *= 2.0 ** -20
    x[5, 7] = 2.0 ** 10
    xt = torch.from_numpy(x).to(torch.bfloat16)
    bits = xt.view(torch.int16).numpy().view(np.uint16)
    ids_ref, wts_ref, margin = oracle.route(bits, inp.router_w, inp.router_bias, wl.k, wl.route_scale)
    ok = margin >= oracle.MARGIN_MIN
    assert ok.sum() >= 4
    out, ids, w = run_few(layer, xt.to(device()))
    y_ref = oracle.layer(bits, ids_ref, wts_ref, inp.experts, inp.shared, wl.swiglu_limit)
    got = bf16_to_f64(out)
    assert np.all(got[0] == 0)
    for t in np.nonzero(ok)[0]:
        assert np.array_equal(ids[t], ids_ref[t])
        if t:
            assert_close(got[t:t + 1], y_ref[t:t + 1], f"token {t}")


def test_tokens_do_not_touch_each_other():
    """A token's row is the same alone and in any company (bit for bit), NaN in another token included."""
    wl, inp, ids, wts, layer = case("medium", 8)
    x = x_to_device(inp.x)
    full = layer.forward_few(x)
    for t in (0, 3, 7):
        assert torch.equal(layer.forward_few(x[t:t + 1].contiguous())[0], full[t])
    bad = x.clone()
    bad[2] = float("nan")
    out = layer.forward_few(bad)
    keep = [t for t in range(8) if t != 2]
    assert torch.equal(out[keep], full[keep]) and torch.isnan(out[2]).all()
    layer.check()


def test_agrees_with_forward_and_leaves_it_alone():
    wl, inp, ids, wts, layer = case("medium", 8)
    x = x_to_device(inp.x)
    y = layer.forward(x)
    few = layer.forward_few(x)
    assert torch.equal(layer.forward(x), y)
    # the same arithmetic but for the fp16 rounding of moe_forward's rows and the order of fp32 sums
    assert_close(bf16_to_f64(few), bf16_to_f64(y), "forward_few against forward")


def test_graph_replay_and_side_stream():
    wl, inp, ids, wts, layer = case("tiny", 4)
    x = x_to_device(inp.x)
    want = layer.forward_few(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = torch.zeros_like(x)
        layer.forward_few(x, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer.forward_few(x, out=out)
        out.zero_()
        for _ in range(3):
            graph.replay()
    side.synchronize()
    assert torch.equal(out, want)


def test_bad_token_ids_are_reported():
    from block_scaled_fp4_sqrt_gb300 import MoEError
    wl, inp, ids, wts, layer = case("hash512", 3)
    x = x_to_device(inp.x)
    good = layer.forward_few(x, token_ids=layer.token_ids)
    tok = layer.token_ids.clone()
    tok[1] = -1
    out = layer.forward_few(x, token_ids=tok)
    with pytest.raises(MoEError):
        layer.check()
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


def test_repeated_table_entries_count_as_often_as_they_stand():
    wl, inp, ids, wts, layer = case("tiny", 2)
    from block_scaled_fp4_sqrt_gb300 import DeviceExperts, MoELayer
    table = torch.tensor([[3, 3], [1, 5]], dtype=torch.int32, device=device())
    lay = MoELayer(wl.d, wl.f, wl.E, wl.k, layer.experts, layer.shared_w, None, None, table, max_T=2, device=device())
    x = x_to_device(inp.x)
    out = lay.forward_few(x, token_ids=torch.tensor([0, 1], dtype=torch.int32, device=device()))
    ids2, w2 = np.array([[3, 3], [1, 5]], np.int32), np.full((2, 2), 0.75)
    y_ref = oracle.layer(inp.x, ids2, w2, inp.experts, inp.shared, wl.swiglu_limit)
    assert_close(bf16_to_f64(out), y_ref, "repeated ids")


def test_bounded_waits_report_a_timeout_and_the_next_call_works():
    import block_scaled_fp4_sqrt_gb300 as moe
    wl, inp, ids, wts, layer = case("tiny", 3)
    x = x_to_device(inp.x)
    want = layer.forward_few(x)
    layer.check()
    moe.moe_set_wait_budget(layer.h, 20_000_000)
    moe.moe_testing_stall_loads(layer.h, True)
    layer.forward_few(x)
    with pytest.raises(moe.MoEError) as err:
        layer.check()
    assert err.value.status == 6
    moe.moe_testing_stall_loads(layer.h, False)
    moe.moe_set_wait_budget(layer.h, 2_000_000_000)
    assert torch.equal(layer.forward_few(x), want)
    layer.check()


def test_refusals():
    import block_scaled_fp4_sqrt_gb300 as moe
    from block_scaled_fp4_sqrt_gb300 import MoELayer
    wl, inp, ids, wts, layer = case("tiny", 8)
    x = x_to_device(inp.x)
    with pytest.raises(moe.MoEError) as err:  # more rows than it takes
        layer2 = MoELayer.from_host(inp, device=device(), max_T=16)
        layer2.forward_few(torch.cat([x, x[:1]]))
    assert err.value.status == 2
    with pytest.raises(moe.MoEError) as err:  # another activation format
        MoELayer.from_host(inp, device=device(), max_T=8, act="mxfp4").forward_few(x)
    assert err.value.status == 2
    with pytest.raises(moe.MoEError) as err:  # token ids without a table
        layer.forward_few(x, token_ids=torch.zeros(8, dtype=torch.int32, device=device()))
    assert err.value.status == 1
    assert layer.forward_few(x[:0]).shape == (0, wl.d)
