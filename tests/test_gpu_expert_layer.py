"""The example's expert layer: its training step against torch's autograd in
float64, its serving path against the decoded 4-bit weights.

Bounds, as shares of a result's 2-norm: a BF16 rounding adds at most 2^-8 of each
value, and the terms of a product keep that share; the longest chain without the
8-bit values has four (dispatch copies, so: pre-activation, SwiGLU, down product,
combine).  E4M3 keeps three bits after the leading one, at most 2^-4 of a value;
values below 2^-14 of their block's largest add less than 2^-17 of that.  SwiGLU's
gradient by one input varies with it by a factor below 2, so a gradient through
the 8-bit values is within 2 * 2^-4 of its norm plus its own four roundings."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer as ex  # noqa: E402
import moe_token_block_amd as m  # noqa: E402

from gpu_util import require_gpu  # noqa: E402

pytestmark = pytest.mark.gpu

ROUNDINGS = 4 * 2.0 ** -8
EIGHT_BITS = 2 * 2.0 ** -4 + ROUNDINGS


def _routing(t, e, k, dev):
    top = torch.topk(torch.randn(t, e, device=dev), k)
    ids = top.indices.int()
    ids[::5, -1] = -1
    w = torch.softmax(top.values, 1)
    return ids.contiguous(), w.contiguous()


def _off(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


def _reference(x, ids, w, w1, w2):
    out = torch.zeros(x.shape[0], w2.shape[1], dtype=x.dtype, device=x.device)
    for j in range(ids.shape[1]):
        for e in range(w1.shape[0]):
            at = (ids[:, j] == e).nonzero()[:, 0]
            a, b = (x[at] @ w1[e].T).chunk(2, 1)
            out = out.index_add(0, at, w[at, j, None] * ((torch.nn.functional.silu(a) * b) @ w2[e].T))
    return out


@pytest.mark.parametrize("t,h,f,e,k", [(70, 128, 64, 5, 2), (256, 320, 96, 4, 3)])
def test_training_step(t, h, f, e, k):
    dev = require_gpu()
    torch.manual_seed(t)
    print(f"training step {t} x {h}", flush=True)
    layer = ex.ExpertLayer(e, h, f, dev, seed=t)
    ids, w = _routing(t, e, k, dev)
    x, dout = torch.randn(t, h, device=dev).bfloat16(), torch.randn(t, h, device=dev).bfloat16()
    out, kept = layer.forward(x, ids, w)
    dx, dw, dw1, dw2 = layer.backward(dout, kept)
    leaves = [v.double().requires_grad_(True) for v in (x, w, layer.w1, layer.w2)]
    want = _reference(leaves[0], ids, leaves[1], leaves[2], leaves[3])
    want.backward(dout.double())
    assert _off(out, want.detach()) <= ROUNDINGS
    assert _off(dw, leaves[1].grad) <= ROUNDINGS
    assert _off(dx, leaves[0].grad) <= EIGHT_BITS
    assert _off(dw1, leaves[2].grad) <= EIGHT_BITS
    assert _off(dw2, leaves[3].grad) <= EIGHT_BITS
    assert not dw[ids < 0].any()


@pytest.mark.parametrize("t", [1, 6, 40])
def test_serving(t):
    dev = require_gpu()
    torch.manual_seed(100 + t)
    h, f, e, k = 256, 128, 4, 2
    print(f"serving {t}", flush=True)
    layer = ex.ExpertLayer(e, h, f, dev, seed=t)
    packed = layer.pack()
    ids, w = _routing(t, e, k, dev)
    x = torch.randn(t, h, device=dev).bfloat16()
    got = ex.serve(x, ids, w, packed, m.ep_entry_plan(t, k, dev))
    w1, w2 = (m.ep_nvfp4_unpack(p.view(-1, p.shape[2]), n).view(e, -1, n).double() for p, n in zip(packed, (h, f)))
    assert _off(got, _reference(x.double(), ids, w.double(), w1, w2)) <= ROUNDINGS
