"""The example's block (residual, norm, expert layer) and its prompt path on the
grouped products: gradients against torch's autograd in float64, 4-bit serving
against the decoded weights, everything in a captured graph.

Bounds, as shares of a result's 2-norm, as for the expert layer: a BF16 rounding adds
at most 2^-8 of each value, E4M3 2^-4.  The references take the values that the 8-bit and 4-bit bytes stand for wherever the
calls take them, so only roundings behind those count."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer as ex  # noqa: E402
import moe_token_block_amd as m  # noqa: E402

from gpu_util import require_gpu  # noqa: E402
from test_gpu_expert_layer import _reference, _routing  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, E4M3 = 2.0 ** -8, 2.0 ** -4


def _off(got, want):
    """The difference as a share of the reference's norm; of a reference that is zeros
    (a token whose only slot is dropped) the result's own norm: no share of 0 is
    anything, and zeros are what a call without terms has to give."""
    norm = float(want.double().norm())
    return float((got.double() - want.double()).norm()) / (norm if norm > 0 else 1.0)


def _inputs(t, h, f, e, k, dev):
    torch.manual_seed(t)
    layer = ex.ExpertLayer(e, h, f, dev, seed=t)
    ids, w = _routing(t, e, k, dev)
    x, res, dout, dh = (torch.randn(t, h, device=dev).bfloat16() for _ in range(4))
    norm = (1 + 0.2 * torch.randn(h, device=dev)).bfloat16()
    return layer, ids, w, x, res, dout, dh, norm


@pytest.mark.parametrize("t,h,f,e,k", [(70, 128, 64, 5, 2), (256, 320, 96, 4, 3), (1, 64, 32, 3, 1)])
def test_block_and_its_gradients(t, h, f, e, k):
    dev = require_gpu()
    print(f"block {t} x {h}", flush=True)
    layer, ids, w, x, res, dout, dh, norm = _inputs(t, h, f, e, k, dev)
    out, total, kept = ex.block_forward(layer, x, res, norm, ids, w)
    dx, dnorm, dw, dw1, dw2 = ex.block_backward(layer, dout, dh, norm, kept)
    hv = (x.float() + res.float()).bfloat16()
    assert torch.equal(total, hv)
    # the layer's part, from the 8-bit rows' values
    rstd = torch.rsqrt(hv.double().square().mean(1, keepdim=True) + 1e-6)
    y = hv.double() * rstd * norm.double()
    data, scales, _, _ = m.rmsnorm_mxfp8(x, norm, res)
    y8 = m.ep_mxfp8_unpack(data, scales).double()
    # E4M3: 2^-4 of a value, and below 2^-6 of a block's unit steps of 2^-9, at most 2^-10 of
    # 2^-8 of the block's largest
    assert _off(y8, y) <= E4M3 + 2.0 ** -16
    leaves = [v.double().requires_grad_(True) for v in (y8, w, layer.w1, layer.w2)]
    want = _reference(leaves[0], ids, *leaves[1:])
    want.backward(dout.double())
    assert _off(out, want.detach()) <= 4 * BF16
    eight = 2 * E4M3 + 4 * BF16  # SwiGLU's gradient from its 8-bit checkpoint
    for got, leaf in ((dw, leaves[1]), (dw1, leaves[2]), (dw2, leaves[3])):
        assert _off(got, leaf.grad) <= eight
    # the norm's part, by autograd from the layer's own gradient of its rows
    dy, _, _, _ = layer.backward(dout, kept[0])
    hl, nl = hv.double().requires_grad_(True), norm.double().requires_grad_(True)
    yn = hl * torch.rsqrt(hl.square().mean(1, keepdim=True) + 1e-6) * nl
    ((yn * dy.double()).sum() + (hl * dh.double()).sum()).backward()
    assert _off(dx, hl.grad) <= 2 * BF16
    assert _off(dnorm, nl.grad) <= 2.0 ** -16


@pytest.mark.parametrize("t", [1, 40, 300])
def test_a_prompt_from_four_bit_weights(t):
    dev = require_gpu()
    print(f"prompt {t}", flush=True)
    h, f, e, k = 256, 128, 4, 2
    layer, ids, w, x, res, _, _, norm = _inputs(t, h, f, e, k, dev)
    packed = layer.pack_mxfp4()
    got, total = ex.serve_prompt(x, res, norm, ids, w, packed)
    assert torch.equal(total, (x.float() + res.float()).bfloat16())
    w1, w2 = (m.ep_mxfp4_unpack(c.view(-1, c.shape[2]), s.view(-1, s.shape[2])).view(c.shape[0], c.shape[1], -1).double()
              for c, s in packed)
    data, scales, _, _ = m.rmsnorm_mxfp8(x, norm, res)
    y = m.ep_mxfp8_unpack(data, scales).double()
    # between the products the rows are rounded to 8 bits once more; the products' own
    # cut of 2^-10 of the terms' magnitudes, sqrt(n) of a sum's size for n random ones
    assert _off(got, _reference(y, ids, w.double(), w1, w2)) <= E4M3 + 4 * BF16 + 2 * 2.0 ** -10 * 16


def test_a_block_in_a_graph():
    """Training step and prompt captured together and replayed with other inputs, other
    routings among them, against eager calls."""
    dev = require_gpu()
    layer, ids, w, x, res, dout, dh, norm = _inputs(96, 128, 64, 5, 2, dev)
    packed = layer.pack_mxfp4()

    def run():
        out, total, kept = ex.block_forward(layer, x, res, norm, ids, w)
        return [out, total, *ex.block_backward(layer, dout, dh, norm, kept), *ex.serve_prompt(x, res, norm, ids, w, packed)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for turn in range(4):
        other, weights = _routing(96, 5, 2, dev)
        ids.copy_(other)
        w.copy_(weights)
        x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, run())):
            assert torch.equal(a, b), (turn, i)
