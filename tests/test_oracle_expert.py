"""The float64 oracle of the expert layer's steps against differences, torch's
autograd in float64 and brute force (CPU)."""

import numpy as np
import pytest
import torch

from oracle import expert, formats as F, mxfp8, nvfp4
from oracle.routing import route_plan


def _routing(rng, t, e, k, drop):
    ids = np.argsort(rng.standard_normal((t, e)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random(ids.shape) < drop] = -1
    return ids


@pytest.mark.parametrize("t,e,k,h,drop", [(5, 4, 2, 7, 0.0), (9, 3, 3, 16, 0.4), (1, 2, 1, 1, 1.0)])
def test_combine_gradients_against_differences_and_autograd(t, e, k, h, drop):
    rng = np.random.default_rng(t)
    plan = route_plan(_routing(rng, t, e, k, drop), e, 16)
    dst = plan["dst_row"]
    rows = rng.standard_normal((len(plan["src_row"]), h))
    w, dout = rng.standard_normal((t, k)), rng.standard_normal((t, h))
    drows, dw, _ = expert.combine_bwd(dout, rows, dst, w)
    loss = lambda r, v: float((dout * expert.combine(r, dst, v)[0]).sum())
    # the loss is linear in each argument: central differences are exact but for rounding
    for i in range(t):
        for j in range(k):
            d = np.zeros_like(w); d[i, j] = 0.5
            assert abs(loss(rows, w + d) - loss(rows, w - d) - dw[i, j]) < 1e-11
    for g in rng.integers(0, rows.shape[0], 20):
        c = rng.integers(0, h)
        d = np.zeros_like(rows); d[g, c] = 0.5
        assert abs(loss(rows + d, w) - loss(rows - d, w) - drows[g, c]) < 1e-11
    r, v = torch.tensor(rows, requires_grad=True), torch.tensor(w, requires_grad=True)
    at, used = torch.tensor(np.maximum(dst, 0)).long(), torch.tensor(dst >= 0)
    ((r[at] * (v * used)[:, :, None]).sum(1) * torch.tensor(dout)).sum().backward()
    np.testing.assert_allclose(drows, r.grad.numpy(), atol=1e-12)
    np.testing.assert_allclose(dw, v.grad.numpy(), atol=1e-11)


def test_dispatch_and_its_gradient():
    rng = np.random.default_rng(3)
    plan = route_plan(_routing(rng, 11, 5, 2, 0.2), 5, 16)
    x = rng.standard_normal((11, 6))
    g = rng.standard_normal((len(plan["src_row"]), 6))
    out = expert.dispatch(x, plan["src_row"])
    for t in range(11):
        for d in plan["dst_row"][t]:
            assert d < 0 or np.array_equal(out[d], x[t])
    assert not out[plan["src_row"] < 0].any()
    dx, _ = expert.combine(g, plan["dst_row"])          # <g, dispatch(x)> = <dx, x>
    assert abs((g * out).sum() - (dx * x).sum()) < 1e-11


def test_matvec_against_the_decoded_matrix():
    rng = np.random.default_rng(4)
    E, N, K = 3, 5, 128
    w = nvfp4.pack_rows(F.f32_to_bf16(rng.standard_normal((E * N, K)).astype(np.float32))).reshape(E, N, -1)
    x = rng.standard_normal((4, K))
    ids = np.array([[0, 2], [1, -1], [2, 0], [-1, -1]], dtype=np.int32)
    y, mag = expert.matvec(x, w, ids)
    for t in range(4):
        for j in range(2):
            want = nvfp4.decode_exact(w[ids[t, j]], K) @ x[t] if ids[t, j] >= 0 else np.zeros(N)
            np.testing.assert_allclose(y[t, j], want, atol=1e-12)
    assert np.all(mag >= np.abs(y) - 1e-12)
    per = np.repeat(x[:, None], 2, axis=1)
    np.testing.assert_array_equal(expert.matvec(per, w, ids)[0], y)
    np.testing.assert_allclose(expert.matvec(x, w[1])[0][1], y[1, 0], atol=1e-12)


def test_swiglu_gradient_against_differences_and_autograd():
    rng = np.random.default_rng(5)
    p, dy = rng.standard_normal((4, 12)) * 3, rng.standard_normal((4, 6))
    g = expert.swiglu_grad(p, dy)
    h = 1e-5
    for i in range(4):
        for c in range(12):
            d = np.zeros_like(p); d[i, c] = h
            diff = ((expert.swiglu(p + d) - expert.swiglu(p - d)) * dy).sum() / (2 * h)
            assert abs(diff - g[i, c]) < 1e-8          # h^2 |f'''| / 6 and 2^-53 |f| / h
    t = torch.tensor(p, requires_grad=True)
    (torch.nn.functional.silu(t[:, :6]) * t[:, 6:] * torch.tensor(dy)).sum().backward()
    np.testing.assert_allclose(g, t.grad.numpy(), atol=1e-13)


def test_checkpoint_values_are_near_their_inputs():
    rng = np.random.default_rng(6)
    bits = F.f32_to_bf16(rng.standard_normal((3, 64)).astype(np.float32))
    v, x = expert.checkpoint_values(bits), expert.f64(bits)
    top = np.repeat(np.abs(x).reshape(3, 2, 32).max(2), 32, axis=1)
    # half a step of three mantissa bits, and below the smallest normal (2^-14 of the block's largest) half of its step
    assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, top * 2.0 ** -17))
    data, scales = mxfp8.pack_rows(bits)
    np.testing.assert_array_equal(v, mxfp8.decode(data, scales))
