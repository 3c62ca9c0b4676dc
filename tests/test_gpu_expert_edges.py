"""The expert layer's calls at their edges on the GPU: empty batches."""

import os
import sys

import numpy as np
import pytest
import torch

import moe_token_block_amd as mtb

from gpu_util import require_gpu, host
from test_gpu_expert import _weights

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
