"""The float64 oracle of the grouped products and the norm against differences,
brute force and torch's autograd in float64 (CPU)."""

import numpy as np
import torch

from oracle import formats as F, mxfp8, products
from oracle.routing import route_plan


def _plan(rng, t, e, k, drop):
    ids = np.argsort(rng.standard_normal((t, e)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random(ids.shape) < drop] = -1
    return ids, route_plan(ids, e, 16)


def test_grouped_products_and_gradients():
    rng = np.random.default_rng(0)
    ids, p = _plan(rng, 9, 4, 2, 0.3)
    n, k, r = 5, 7, len(p["src_row"])
    x, w, d = rng.standard_normal((9, k)), rng.standard_normal((4, n, k)), rng.standard_normal((r, n))
    rows = np.where(p["src_row"][:, None] >= 0, x[np.maximum(p["src_row"], 0)], np.nan)
    d[p["src_row"] < 0] = np.nan
    out, _ = products.gemm(rows, w, p["counts"], p["offsets"])
    for t in range(9):
        for j in range(2):
            if ids[t, j] >= 0:
                np.testing.assert_allclose(out[p["dst_row"][t, j]], w[ids[t, j]] @ x[t], rtol=1e-13)
    assert not out[p["src_row"] < 0].any()
    # <d, out> has these gradients; it is linear in rows and in w: differences are exact but for rounding
    used = p["src_row"] >= 0
    loss = lambda a, b: float((d[used] * products.gemm(a, b, p["counts"], p["offsets"])[0][used]).sum())  # noqa: E731
    drows, _ = products.dgrad(d, w, p["counts"], p["offsets"])
    dw, _ = products.wgrad(d, rows, p["counts"], p["offsets"])
    assert not drows[~used].any()
    for g in np.nonzero(used)[0]:
        c = int(rng.integers(0, k))
        u = np.zeros_like(rows); u[g, c] = 0.5
        assert abs(loss(rows + u, w) - loss(rows - u, w) - drows[g, c]) < 1e-11
    for _ in range(20):
        i = tuple(int(rng.integers(0, s)) for s in w.shape)
        u = np.zeros_like(w); u[i] = 0.5
        assert abs(loss(rows, w + u) - loss(rows, w - u) - dw[i]) < 1e-11


def test_norm_against_autograd_and_differences():
    rng = np.random.default_rng(1)
    t, h, eps = 4, 64, 1e-5
    x, w, dy, dh = (rng.standard_normal(s) for s in ((t, h), (h,), (t, h), (t, h)))
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = tx * torch.rsqrt(tx.square().mean(1, keepdim=True) + eps) * tw
    ((y * torch.tensor(dy)).sum() + (tx * torch.tensor(dh)).sum()).backward()
    rstd, want = products.rmsnorm(x, w, eps)
    np.testing.assert_allclose(want, y.detach().numpy(), rtol=1e-13)
    dx, dw = products.drmsnorm(dy, x, w, rstd, dh)
    np.testing.assert_allclose(dx, tx.grad.numpy(), atol=1e-13)
    np.testing.assert_allclose(dw, tw.grad.numpy(), atol=1e-12)
    loss = lambda a: float((dy * products.rmsnorm(a, w, eps)[1]).sum() + (dh * a).sum())  # noqa: E731
    for _ in range(10):
        i = (int(rng.integers(0, t)), int(rng.integers(0, h)))
        u = np.zeros_like(x); u[i] = 1e-5
        assert abs((loss(x + u) - loss(x - u)) / 2e-5 - dx[i]) < 1e-8


def test_mxfp8_of_fp32_rows():
    rng = np.random.default_rng(2)
    bits = F.f32_to_bf16((rng.standard_normal((6, 96)) * np.exp2(rng.integers(-130, 120, (6, 1)))).astype(np.float32))
    want = mxfp8.pack_rows(bits)
    got = products.mxfp8_f32(F.bf16_to_f32(bits))
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    y = np.ones((1, 64), dtype=np.float32)
    y[0, 3] = np.inf
    assert products.mxfp8_f32(y)[1].tolist() == [[255, 119]]  # 1 = 256 * 2^-8: the least e with 1 <= 448 * 2^e is -8
    y = np.array([[1.0 + 2.0 ** -4] + [448.0] + [0.0] * 30], dtype=np.float32)
    d, s = products.mxfp8_f32(y)
    assert s[0, 0] == 127 and d[0, 0] == 0x38 and d[0, 1] == 0x7E  # the tie between 1 and 1.125 goes to the even one
