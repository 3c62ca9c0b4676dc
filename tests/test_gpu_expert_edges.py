"""The expert layer's calls at their edges on the GPU: empty batches, weights of
unused slots that are not numbers, pre-activations that are not finite, small
weights times large activations, one plan in a captured graph, no autograd graph.
Bounds are those of ``test_gpu_expert``."""

import os
import sys

import numpy as np
import pytest
import torch

import moe_token_block_amd as mtb
from oracle import expert, mxfp8, nvfp4

from gpu_util import require_gpu, bf16_dev, host, assert_bytes_equal
from test_gpu_expert import U, _act_slack, _bits, _check_matvec, _grad_slack, _ids, _near, _plan, _weights

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


# ------------------------------------------------------------------ empty batches
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("per_entry", [False, True])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_matvec_of_no_tokens(dev, swiglu, per_entry, idt):
    e, k, n, h = 4, 2, 6, 128
    weight = torch.from_numpy(_weights(np.random.default_rng(0), e, n, h)).to(dev)
    ids = torch.zeros((5, k), dtype=idt, device=dev)
    x = torch.zeros((5, k, h) if per_entry else (5, h), dtype=torch.bfloat16, device=dev)
    got = mtb.ep_nvfp4_expert_matvec(x[:0], weight, ids[:0], swiglu=swiglu)
    assert got.shape == (0, k, n // 2 if swiglu else n) and got.dtype == torch.bfloat16


def test_serving_no_tokens(dev):
    layer = ex.ExpertLayer(4, 128, 64, dev)
    ids, w = torch.zeros((0, 2), dtype=torch.int32, device=dev), torch.zeros((0, 2), device=dev)
    x = torch.zeros((0, 128), dtype=torch.bfloat16, device=dev)
    assert ex.serve(x, ids, w, layer.pack(), mtb.ep_entry_plan(0, 2, dev)).shape == (0, 128)
    # the other calls of the layer on no tokens
    plan = mtb.ep_route_plan(ids, 4)
    rows = mtb.ep_bf16_dispatch(x, plan)
    assert mtb.ep_bf16_combine(rows, plan, w).shape == (0, 128)
    drows, dw = mtb.ep_bf16_combine_bwd(x, rows, plan, w)
    assert dw.shape == (0, 2) and not host(drows).any()
    act, data, scales = mtb.swiglu_mxfp8_checkpoint(x)
    dx, act2 = mtb.dswiglu_mxfp8_checkpoint(data, scales, act)
    assert dx.shape == (0, 128) and act2.shape == act.shape == (0, 64)
    assert mtb.ep_mxfp8_unpack(data, scales).shape == (0, 128)


# ------------------------------------------------------------------ unused slots
@pytest.mark.parametrize("idt", [np.int32, np.int64])
@pytest.mark.parametrize("t,e,k,h", [(1, 4, 2, 4096), (6, 4, 2, 5), (9, 12, 9, 7), (40, 3, 1, 8), (33, 6, 2, 521),
                                     (21, 16, 8, 1024), (70, 5, 3, 1001)])
def test_combine_of_entries_with_unused_slots(dev, idt, t, e, k, h):
    # the entries' plan names every slot: those whose id names no expert add nothing, whatever their weight and row hold
    rng = np.random.default_rng(t * h + k)
    ids = _ids(rng, t, e, k, 0.4).astype(idt)
    ids[0, 0] = e                                             # no expert, nor is -2 or (64 bits) 2^32
    ids[-1, -1] = -2 if idt is np.int32 else 2 ** 32
    used = (ids >= 0) & (ids < e)
    rows, w = _bits(rng.standard_normal((t * k, h))), rng.standard_normal((t, k)).astype(np.float32)
    rows[~used.reshape(-1)] = 0x7FC0
    w[~used] = rng.choice([np.nan, np.inf, -np.inf], size=(~used).sum())
    dst = np.where(used, np.arange(t * k).reshape(t, k), -1).astype(np.int32)
    rd, wd, idd = bf16_dev(rows, dev), torch.from_numpy(w).to(dev), torch.from_numpy(ids).to(dev)
    entries = mtb.ep_entry_plan(t, k, dev)
    got = mtb.ep_bf16_combine(rd, entries, wd, topk_idx=idd, num_experts=e)
    want, mag = expert.combine(expert.f64(rows), dst, w)
    _near(got, want, (k + 1) * U * mag, "weighted")
    marked = dict(entries, dst_row=torch.from_numpy(dst).to(dev))
    assert_bytes_equal(host(got), host(mtb.ep_bf16_combine(rd, marked, wd)), "a plan that marks them")
    want, mag = expert.combine(expert.f64(rows), dst)
    _near(mtb.ep_bf16_combine(rd, entries, topk_idx=idd, num_experts=e), want, (k + 1) * U * mag, "without weights")


def test_combine_takes_both_the_plans_marks_and_the_ids(dev):
    rng = np.random.default_rng(2)
    t, e, k, h = 19, 5, 2, 72
    ids = _ids(rng, t, e, k, 0.3)
    plan = _plan(ids, e, 16, dev)
    fewer = np.where(rng.random(ids.shape) < 0.3, -1, np.abs(ids)).astype(np.int32)  # |-1| = 1 names an expert again
    dst = np.where(fewer >= 0, host(plan["dst_row"]), -1)
    rows, w = _bits(rng.standard_normal((plan["r_cap"], h))), rng.standard_normal((t, k)).astype(np.float32)
    w[dst < 0] = np.nan
    got = mtb.ep_bf16_combine(bf16_dev(rows, dev), plan, torch.from_numpy(w).to(dev),
                              topk_idx=torch.from_numpy(fewer).to(dev), num_experts=e)
    want, mag = expert.combine(expert.f64(rows), dst, w)
    _near(got, want, (k + 1) * U * mag, "combine")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_serving_with_a_weight_that_is_no_number_in_an_unused_slot(dev, bad):
    torch.manual_seed(3)
    t, h, f, e, k = 5, 256, 128, 4, 2
    layer = ex.ExpertLayer(e, h, f, dev, seed=1)
    x = torch.randn(t, h, device=dev).bfloat16()
    top = torch.topk(torch.randn(t, e, device=dev), k)
    ids, w = top.indices.int(), torch.softmax(top.values, 1)
    ids[1] = -1                                               # a token with no expert at all
    ids[3, 1] = -1
    clean = w.masked_fill(ids < 0, 0.0)
    packed, entries = layer.pack(), mtb.ep_entry_plan(t, k, dev)
    got = ex.serve(x, ids, w.masked_fill(ids < 0, bad), packed, entries)
    assert_bytes_equal(host(got), host(ex.serve(x, ids, clean, packed, entries)), "served")
    assert not host(got)[1].any() and bool(torch.isfinite(got.float()).all())
    # as the training path has it
    out, _ = layer.forward(x, ids, w.masked_fill(ids < 0, bad))
    assert not host(out)[1].any() and bool(torch.isfinite(out.float()).all())


def test_combine_refuses_ids_that_do_not_fit(dev):
    rows = torch.zeros((6, 16), dtype=torch.bfloat16, device=dev)
    entries = mtb.ep_entry_plan(3, 2, dev)
    ids = torch.zeros((3, 2), dtype=torch.int32, device=dev)
    for kw in (dict(topk_idx=ids), dict(topk_idx=ids[:2], num_experts=4), dict(topk_idx=ids.cpu(), num_experts=4),
               dict(topk_idx=ids.float(), num_experts=4), dict(topk_idx=ids.view(6), num_experts=4),
               dict(topk_idx=ids.t().contiguous().t(), num_experts=4), dict(topk_idx=ids, num_experts=0),
               dict(topk_idx=ids, num_experts=1025)):
        with pytest.raises((ValueError, TypeError, mtb.EpError)):
            mtb.ep_bf16_combine(rows, entries, **kw)
            raise AssertionError(f"{kw} was not refused")


# ------------------------------------------------------------------ pre-activations that are not finite
@pytest.mark.parametrize("t,f", [(1, 32), (4, 96), (9, 1024)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), -float("nan")])
def test_checkpoint_of_a_block_that_is_not_finite(dev, t, f, bad):
    # such a block of 32 comes back as NaN, whole, so that the gradient shows what the output does; the others keep
    # their bytes
    rng = np.random.default_rng(t + f)
    p = rng.standard_normal((t, 2 * f)).astype(np.float32) * 3
    p[0, 0:32] = 0.0                                          # a block of zeros but for the one value
    clean = _bits(p)
    p[0, 5] = bad                                             # in a gate
    p[-1, f + 31] = bad                                       # and in an up value
    where = np.zeros((t, 2 * f), dtype=bool)
    where[0, 0:32] = where[-1, f : f + 32] = True
    pb, dyb = _bits(p), _bits(rng.standard_normal((t, f)))
    pb[0, 5] = np.uint16(torch.tensor(bad).bfloat16().view(torch.int16).item() & 0xFFFF)
    pb[-1, f + 31] = pb[0, 5]
    act, data, scales = mtb.swiglu_mxfp8_checkpoint(bf16_dev(pb, dev))
    wd, ws = mxfp8.pack_rows(clean)
    blocks = where[:, ::32]
    assert np.all(host(scales)[blocks] == 255)
    assert_bytes_equal(host(scales)[~blocks], ws[~blocks], "scales of the other blocks")
    assert_bytes_equal(host(data)[~where], wd[~where], "data of the other blocks")
    back = host(mtb.ep_mxfp8_unpack(data, scales))
    assert np.all((back[where] & 0x7FFF) > 0x7F80) and np.all((back[~where] & 0x7F80) < 0x7F80)
    # the output follows the formula value by value
    a = expert.f64(clean)
    want, slack = expert.swiglu(a), _act_slack(a)
    hit = np.zeros((t, f), dtype=bool)
    hit[0, 5] = hit[-1, 31] = True
    got = host(act).copy()
    assert np.all((got[hit] & 0x7FFF) >= 0x7F80)
    got[hit] = host(mtb.swiglu_mxfp8_checkpoint(bf16_dev(clean, dev))[0])[hit]
    _near(got, want, slack, "act")
    # the gradient: NaN wherever the block is an argument (db = dy * silu(a) has none of b's), the formula elsewhere
    dx, act2 = mtb.dswiglu_mxfp8_checkpoint(data, scales, bf16_dev(dyb, dev))
    lost = where[:, :f] | where[:, f:]
    dxn, actn = np.isnan(expert.f64(host(dx))), np.isnan(expert.f64(host(act2)))
    np.testing.assert_array_equal(actn, lost)
    np.testing.assert_array_equal(dxn, np.concatenate([lost, where[:, :f]], 1))
    v, dy = mxfp8.decode(wd, ws), expert.f64(dyb)
    got = host(dx).copy()
    want, slack = expert.swiglu_grad(v, dy), _grad_slack(v, dy)
    got[dxn] = _bits(want)[dxn]
    _near(got, want, slack, "dx")


# ------------------------------------------------------------------ small weights, large activations
# tokens, experts, width, hidden: a block's few rows, blocks of more waves, and the kernel for many entries
@pytest.mark.parametrize("t,e,n,k", [(3, 1, 24, 192), (70, 20, 514, 128), (288, 16, 2050, 64)])
@pytest.mark.parametrize("scale,x_scale", [(2.0 ** -62, 2.0 ** 126), (2.0 ** -55, 2.0 ** 126), (2.0 ** -22, 2.0 ** 126),
                                           (2.0 ** -24, 2.0 ** -80), (2.0 ** -110, 2.0 ** 20)])
def test_matvec_of_small_weights_and_large_activations(dev, t, e, n, k, scale, x_scale):
    # sums that are ordinary numbers, or large ones, may not leave FP32's range on the way
    rng = np.random.default_rng(t)
    w = nvfp4.pack_rows(_bits(rng.standard_normal((e * n, k)) * scale)).reshape(e, n, -1)
    xb = _bits(np.clip(rng.standard_normal((t, k)), -1.9, 1.9) * x_scale)
    ids = (rng.permutation(t) % e).astype(np.int32)[:, None]
    print(f"small weights {t} {e} {n} {k} {scale} {x_scale}", flush=True)
    got = mtb.ep_nvfp4_expert_matvec(bf16_dev(xb, dev), torch.from_numpy(w).to(dev), torch.from_numpy(ids).to(dev))
    y, _ = expert.matvec(expert.f64(xb), w, ids)
    assert np.abs(y).max() < 2.0 ** 127
    _check_matvec(got, expert.f64(xb), w, ids, False, f"scale {scale}")


# ------------------------------------------------------------------ graphs, autograd
def test_serving_in_a_graph_follows_its_ids(dev):
    # one plan for every step: what a replay drops are the slots that its ids leave unused
    torch.manual_seed(4)
    t, h, f, e, k = 6, 256, 64, 8, 2
    layer = ex.ExpertLayer(e, h, f, dev, seed=2)
    packed, entries = layer.pack(), mtb.ep_entry_plan(t, k, dev)
    x = torch.randn(t, h, device=dev).bfloat16()
    ids = torch.zeros((t, k), dtype=torch.int32, device=dev)
    w = torch.zeros((t, k), device=dev)

    def step(drop):
        top = torch.topk(torch.randn(t, e, device=dev), k)
        unused = torch.rand(t, k, device=dev) < drop
        ids.copy_(top.indices.int().masked_fill(unused, -1))
        w.copy_(torch.softmax(top.values, 1).masked_fill(unused, float("nan")))
        x.copy_(torch.randn(t, h, device=dev).bfloat16())

    step(0.0)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        ex.serve(x, ids, w, packed, entries)
    torch.cuda.current_stream(dev).wait_stream(side)
    torch.cuda.synchronize(dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ex.serve(x, ids, w, packed, entries)
    for i, drop in enumerate((0.0, 0.5, 1.0, 0.2)):
        step(drop)
        g.replay()
        torch.cuda.synchronize(dev)
        assert_bytes_equal(host(out), host(ex.serve(x, ids, w, packed, entries)), f"replay {i}")
        assert bool(torch.isfinite(out.float()).all()) and not host(out)[host((ids < 0).all(1))].any()


def test_results_carry_no_autograd_graph(dev):
    x = torch.randn(4, 128, device=dev).bfloat16().requires_grad_(True)
    w = torch.rand(4, 2, device=dev).requires_grad_(True)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=dev)
    plan = mtb.ep_route_plan(ids, 2)
    rows = mtb.ep_bf16_dispatch(x, plan)
    act, data, scales = mtb.swiglu_mxfp8_checkpoint(x)
    weight = mtb.ep_nvfp4_pack(torch.randn(8, 128, device=dev).bfloat16()).view(2, 4, -1)
    results = [rows, mtb.ep_bf16_combine(rows, plan, w), *mtb.ep_bf16_combine_bwd(x, rows, plan, w), act,
               mtb.ep_nvfp4_expert_matvec(x, weight, ids), *mtb.dswiglu_mxfp8_checkpoint(data, scales, act)]
    assert not any(r.requires_grad for r in results)
