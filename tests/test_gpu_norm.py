"""The norm with an MXFP8 output and its gradient on the GPU against float64.

Bars, with u = 2^-24: rstd: a sum of H squares in any order is within (H + 1) u of
itself, and the mean, the root, the quotient and eps add four roundings, the first
three halved or not: (H / 2 + 4) u.  h is equal bit for bit; so are the 8-bit
bytes to the oracle's of fl(fl(h rstd) weight) with the call's own rstd.  Gradients:
the sums' bounds carried through the formula, one rounding to BF16 (2^-8) for dx.
"""

import numpy as np
import pytest
import torch

import moe_token_block_amd as mtb
from oracle import formats as F
from oracle import expert, products

from gpu_util import require_gpu, bf16_dev, host, assert_bytes_equal

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# every number of chunks a thread and of threads a row, partly filled ones among them
SHAPES = [(1, 32), (3, 64), (5, 96), (2, 512), (3, 544), (2, 1024), (4, 1056), (7, 2048), (3, 2080), (2, 4096), (5, 4128),
          (2, 7168), (3, 8192), (2, 8224), (2, 16384), (0, 64), (1300, 64), (700, 2048), (600, 4096)]


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _bits(x):
    return F.f32_to_bf16(np.asarray(x, dtype=np.float32))


def _inputs(t, h, seed=0):
    rng = np.random.default_rng(t * h + seed)
    x = rng.standard_normal((t, h)) * np.exp(rng.standard_normal((t, 1)))
    return _bits(x), _bits(rng.standard_normal((t, h))), _bits(1 + 0.2 * rng.standard_normal(h))


def _check(x, res, w, eps, out):
    data, scales, h, rstd = (host(v) for v in out)
    hb = x if res is None else _bits(F.bf16_to_f32(x) + F.bf16_to_f32(res))
    assert_bytes_equal(h, hb, "h")
    want, _ = products.rmsnorm(expert.f64(hb), expert.f64(w), eps)
    assert np.all(np.abs(rstd - want) <= (x.shape[1] / 2 + 4) * U * want), "rstd"
    y = (F.bf16_to_f32(hb) * rstd[:, None]) * F.bf16_to_f32(w)  # FP32, each step rounded
    wd, ws = products.mxfp8_f32(y)
    assert_bytes_equal(scales, ws, "scales")
    assert_bytes_equal(data, wd, "data")


@pytest.mark.parametrize("t,h", SHAPES)
def test_norm(dev, t, h):
    print(f"norm {t} x {h}", flush=True)
    x, r, w = _inputs(t, h)
    xd, rd, wd = (bf16_dev(v, dev) for v in (x, r, w))
    _check(x, r, w, 1e-6, mtb.rmsnorm_mxfp8(xd, wd, rd))
    out = mtb.rmsnorm_mxfp8(xd, wd, eps=1e-5)
    assert out[2] is xd
    _check(x, None, w, 1e-5, out)


def test_norm_of_zero_tiny_and_large_rows(dev):
    h = 256
    x = np.zeros((6, h), dtype=np.float32)
    x[1, :] = 2.0 ** -130
    x[2, 7] = 2.0 ** 60
    x[3, :] = np.where(np.arange(h) % 2, 1.0, -1.0)
    x[4, :] = 2.0 ** np.linspace(-100, 40, h)
    x[5, :32] = 1.0
    w = np.exp2(np.linspace(-120, 3, h))
    for ww in (np.ones(h), w):
        xb, wb = _bits(x), _bits(ww)
        _check(xb, None, wb, 1e-6, mtb.rmsnorm_mxfp8(bf16_dev(xb, dev), bf16_dev(wb, dev)))
        with pytest.raises(mtb.EpError):  # FP32 loses the tiny row's squares: nothing is left to divide by
            mtb.rmsnorm_mxfp8(bf16_dev(xb[1:], dev), bf16_dev(wb, dev), eps=0.0)
        _check(xb, None, wb, 2.0 ** -100, mtb.rmsnorm_mxfp8(bf16_dev(xb, dev), bf16_dev(wb, dev), eps=2.0 ** -100))


def test_norm_of_rows_that_are_not_finite(dev):
    x, r, w = _inputs(4, 96)
    xd = bf16_dev(x, dev)
    xd[1, 40] = float("nan")
    xd[2, 70] = float("inf")
    data, scales, h, rstd = mtb.rmsnorm_mxfp8(xd, bf16_dev(w, dev))
    y = mtb.ep_mxfp8_unpack(data, scales).float().cpu().numpy()
    assert np.isnan(y[1]).all() and np.isnan(y[2, 64:96]).all()
    clean = bf16_dev(x, dev)
    ref = mtb.rmsnorm_mxfp8(clean, bf16_dev(w, dev))
    for i in (0, 3):
        assert torch.equal(data[i], ref[0][i]) and torch.equal(scales[i], ref[1][i])


def test_the_sum_in_place(dev):
    x, r, w = _inputs(9, 4128)
    wd = bf16_dev(w, dev)
    want = mtb.rmsnorm_mxfp8(bf16_dev(x, dev), wd, bf16_dev(r, dev))
    for which in (0, 1):
        xd, rd = bf16_dev(x, dev), bf16_dev(r, dev)
        got = mtb.rmsnorm_mxfp8(xd, wd, rd, h=(xd, rd)[which])
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("t,h", SHAPES)
def test_gradient(dev, t, h, with_dh):
    print(f"gradient {t} x {h} {with_dh}", flush=True)
    x, dh, w = _inputs(t, h, 1)
    dy = _bits(np.random.default_rng(t + h).standard_normal((t, h)))
    rstd = (1 / np.sqrt((expert.f64(x) ** 2).mean(axis=1) + 1e-6)).astype(np.float32)
    args = [bf16_dev(v, dev) for v in (dy, x, w)] + [torch.from_numpy(rstd).to(dev)]
    dx, dw = mtb.drmsnorm(*args, dh=bf16_dev(dh, dev) if with_dh else None)
    y, f, ww, r = expert.f64(dy), expert.f64(x), expert.f64(w), rstd.astype(np.float64)
    d = expert.f64(dh) if with_dh else None
    want, want_w = products.drmsnorm(y, f, ww, r, d)
    g, r = y * ww, r[:, None]
    # the dot product's bound ((H + 2) u of its terms' magnitudes, and the product g before
    # it u), times 1/H, r^2 and h with a rounding each
    kmag = np.abs(g * f).sum(1, keepdims=True) / max(h, 1) * r * r
    slack = r * (np.abs(f) * kmag * (h + 8) * U + 4 * U * (np.abs(g) + np.abs(f) * kmag))
    slack = slack + (0 if d is None else U * np.abs(d))
    got = dx.double().cpu().numpy()
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= slack + 2.0 ** -8 * (np.abs(want) + slack) + 2.0 ** -134), "dx"
    mag = np.abs(y * f * r).sum(0)
    assert dw.shape == (h,) and np.all(np.abs(host(dw) - want_w) <= (t + 3) * U * mag), "dweight"
    again = mtb.drmsnorm(*args, dh=bf16_dev(dh, dev) if with_dh else None)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_streams_graphs_and_addresses(dev):
    x, r, w = _inputs(33, 1056)
    xd, rd, wd = (bf16_dev(v, dev) for v in (x, r, w))

    def run(x, r, w):
        o = mtb.rmsnorm_mxfp8(x, w, r)
        return list(o) + list(mtb.drmsnorm(r, o[2], w, o[3], x))

    want = run(xd, rd, wd)
    odd = []
    for v in (xd, rd, wd):
        b = torch.empty(v.numel() + 1, dtype=v.dtype, device=dev)
        b[1:] = v.reshape(-1)
        odd.append(b[1:].view(v.shape))
    for a, b in zip(run(*odd), want):
        assert torch.equal(a, b)
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(s):
        got = run(xd, rd, wd)
    torch.cuda.current_stream(dev).wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(xd, rd, wd)
    for turn in range(3):
        xd.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, run(xd, rd, wd)):
            assert torch.equal(a, b), turn


def test_refusals(dev):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    f32 = torch.zeros(4, device=dev)
    for call in (lambda: mtb.rmsnorm_mxfp8(bf(4, 48), bf(48)), lambda: mtb.rmsnorm_mxfp8(bf(4, 64), bf(32)),
                 lambda: mtb.rmsnorm_mxfp8(bf(4, 64), bf(64).float()), lambda: mtb.rmsnorm_mxfp8(bf(4, 64), bf(64), bf(3, 64)),
                 lambda: mtb.rmsnorm_mxfp8(bf(4, 64), bf(64), h=bf(4, 64)),
                 lambda: mtb.drmsnorm(bf(4, 64), bf(4, 64), bf(64), f32.double()),
                 lambda: mtb.drmsnorm(bf(4, 64), bf(3, 64), bf(64), f32),
                 lambda: mtb.drmsnorm(bf(40, 64), bf(40, 64), bf(64), torch.zeros(40, device=dev), workspace=torch.zeros(8, dtype=torch.uint8, device=dev))):
        with pytest.raises((ValueError, TypeError)):
            call()
    for call in (lambda: mtb.rmsnorm_mxfp8(bf(1, 16416), bf(16416)), lambda: mtb.rmsnorm_mxfp8(bf(1, 64), bf(64), eps=-1.0),
                 lambda: mtb.rmsnorm_mxfp8(bf(1, 64), bf(64), eps=float("nan"))):
        with pytest.raises(mtb.EpError):
            call()
