"""Every operand of the grouped products, the MXFP4 pack and the norm with bytes past
4 GiB, one operand at a time; rows on both sides of 2^31 and 2^32 bytes and elements.

A far row's results have to be those of the same row handed over alone where the call
takes rows by themselves, and within the bars of the small sizes otherwise (u = 2^-24,
(n + 1) u of the sum of the terms' magnitudes and one BF16 rounding)."""

import pytest
import torch

import moe_token_block_amd as mtb

from gpu_util import require_gpu
from test_gpu_products_large import _near

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
GIB4 = 1 << 32


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    yield d
    torch.cuda.empty_cache()


def _rand(dev, *shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device=dev).manual_seed(seed), device=dev, dtype=torch.bfloat16)


def _bytes(dev, *shape):
    """E4M3 or E2M1 bytes without E4M3's NaN."""
    b = torch.randint(0, 255, shape, generator=torch.Generator(device=dev).manual_seed(1), device=dev, dtype=torch.uint8)
    return b.bitwise_and_(0xF7)


def _at(dev, rows, row_bytes):
    """The first and last row and those around 2^31 and 2^32 bytes, and twice that."""
    at = {0, rows - 1}
    for b in (1 << 31, 1 << 32, 1 << 33):
        at.update(r for r in (b // row_bytes - 1, b // row_bytes, b // row_bytes + 1) if r < rows)
    return torch.tensor(sorted(at), device=dev)


def _values4(codes, scales):
    return mtb.ep_mxfp4_unpack(codes.contiguous(), scales.contiguous()).double()


def _values8(data, scales):
    return mtb.ep_mxfp8_unpack(data.contiguous(), scales.contiguous()).double()


def test_results_of_the_products(dev):
    m, n, k = 270_000, 8192, 32
    print("results", flush=True)
    at = _at(dev, m, 2 * n)
    x, w = _rand(dev, m, k), _rand(dev, n, k, seed=1)
    assert 2 * m * n > GIB4 and m * n > 1 << 31
    y = mtb.ep_bf16_grouped_gemm(x, w)
    a, b = x[at].double(), w.double().T.contiguous()
    _near(y[at], a @ b, (k + 1) * U * (a.abs() @ b.abs()), "gemm")
    del y
    wc, ws = mtb.ep_mxfp4_pack(w)
    b = _values4(wc, ws).T.contiguous()
    for (d, s), values in ((mtb.ep_mxfp4_pack(x), _values4), (mtb.ep_mxfp8_pack(x)[:2], _values8)):
        y = mtb.ep_mxfp4_grouped_gemm(d, s, wc, ws)
        a = values(d[at], s[at])
        _near(y[at], a @ b, (k + 1) * U * (a.abs() @ b.abs()), "mx")
        del y


def test_gradients_of_the_weights_from_far_dout(dev):
    m, n, k = 270_000, 8192, 24
    print("dout", flush=True)
    at = _at(dev, m, 2 * n)
    d, x = _rand(dev, m, n), torch.zeros((m, k), dtype=torch.bfloat16, device=dev)
    x[at] = _rand(dev, len(at), k, seed=2)
    a, b = d[at].double().T.contiguous(), x[at].double()
    _near(mtb.ep_bf16_grouped_wgrad(d, x), a @ b, (len(at) + 1) * U * (a.abs() @ b.abs()), "wgrad")
    w = _rand(dev, n, k, seed=3)
    a, b = d[at].double(), w.double()
    _near(mtb.ep_bf16_grouped_dgrad(d, w)[at], a @ b, (n + 1) * U * (a.abs() @ b.abs()), "dgrad")


def test_eight_and_four_bit_rows(dev):
    k, n = 8192, 24
    wc, ws = mtb.ep_mxfp4_pack(_rand(dev, n, k))
    b = _values4(wc, ws).T.contiguous()
    for rows, row_bytes, values in ((540_000, k, _values8), (1_080_000, k // 2, _values4)):
        print("rows", rows, flush=True)
        assert rows * row_bytes > GIB4
        at = _at(dev, rows, row_bytes)
        d = _bytes(dev, rows, row_bytes)
        s = torch.full((rows, k // 32), 120, dtype=torch.uint8, device=dev)
        s[at] = 125
        y = mtb.ep_mxfp4_grouped_gemm(d, s, wc, ws)
        a = values(d[at], s[at])
        _near(y[at], a @ b, (k + 1) * U * (a.abs() @ b.abs()), "mx")
        del d, s, y


def _room(dev, e, rows):
    """A plan of `rows` rows an expert."""
    i32 = dict(dtype=torch.int32, device=dev)
    return dict(counts=torch.full((e,), rows, **i32), offsets=torch.arange(e + 1, **i32) * rows,
                dst_row=torch.arange(e * rows, **i32).view(-1, 1), src_row=torch.zeros(e * rows, **i32), r_cap=e * rows,
                num_experts=e, alignment=1)


@pytest.mark.parametrize("rows", [2, 40])  # the kernels for few rows, and tiles
def test_weights(dev, rows):
    print("weights", rows, flush=True)
    e, n, k = 140, 4096, 4096
    assert 2 * e * n * k > GIB4
    plan = _room(dev, e, rows)
    w = _rand(dev, e, n, k)
    x, d = _rand(dev, e * rows, k, seed=1), _rand(dev, e * rows, n, seed=2)
    out, dx = mtb.ep_bf16_grouped_gemm(x, w, plan), mtb.ep_bf16_grouped_dgrad(d, w, plan)
    dw = mtb.ep_bf16_grouped_wgrad(d, x, plan)
    dw32 = mtb.ep_bf16_grouped_wgrad(d, x, plan, dtype=torch.float32)
    for i in (0, 63, 64, 127, 128, e - 1):  # 2^25 bytes an expert
        at = slice(i * rows, (i + 1) * rows)
        for got, a, b, terms, step in ((out[at], x[at].double(), w[i].double().T.contiguous(), k, 2.0 ** -8),
                                       (dx[at], d[at].double(), w[i].double(), n, 2.0 ** -8),
                                       (dw[i], d[at].double().T.contiguous(), x[at].double(), rows, 2.0 ** -8),
                                       (dw32[i], d[at].double().T.contiguous(), x[at].double(), rows, U)):
            _near(got, a @ b, (terms + 1) * U * (a.abs() @ b.abs()), (i, terms), step)


@pytest.mark.parametrize("rows", [2, 40])
def test_four_bit_weights(dev, rows):
    print("weights", rows, flush=True)
    e, n, k = 520, 4096, 4096
    assert e * n * k // 2 > GIB4
    plan = _room(dev, e, rows)
    wc = _bytes(dev, e * n, k // 2).view(e, n, k // 2)
    ws = torch.full((e, n, k // 32), 121, dtype=torch.uint8, device=dev)
    ws[:, ::3] = 127
    x = _rand(dev, e * rows, k, seed=1)
    for (d, s), values in ((mtb.ep_mxfp4_pack(x), _values4), (mtb.ep_mxfp8_pack(x)[:2], _values8)):
        y = mtb.ep_mxfp4_grouped_gemm(d, s, wc, ws, plan)
        for i in (0, 255, 256, 511, 512, e - 1):  # 2^23 bytes an expert
            at = slice(i * rows, (i + 1) * rows)
            a, b = values(d[at], s[at]), _values4(wc[i], ws[i]).T.contiguous()
            _near(y[at], a @ b, (k + 1) * U * (a.abs() @ b.abs()), i)


def test_pack_and_unpack(dev):
    rows, h = 300_000, 8192
    print("pack", flush=True)
    at = _at(dev, rows, 2 * h)
    x = _rand(dev, rows, h)
    c, s = mtb.ep_mxfp4_pack(x)
    wc, ws = mtb.ep_mxfp4_pack(x[at])
    assert torch.equal(c[at], wc) and torch.equal(s[at], ws)
    y = mtb.ep_mxfp4_unpack(c, s)
    assert torch.equal(y[at], mtb.ep_mxfp4_unpack(wc, ws))
    del x, y
    rows = 1_100_000  # the codes themselves past 4 GiB
    c = _bytes(dev, rows, h // 2)
    s = torch.full((rows, h // 32), 127, dtype=torch.uint8, device=dev)
    at = _at(dev, rows, h // 2)
    y = mtb.ep_mxfp4_unpack(c, s)
    assert torch.equal(y[at], mtb.ep_mxfp4_unpack(c[at], s[at]))
    c2, s2 = mtb.ep_mxfp4_pack(y)
    wc, ws = mtb.ep_mxfp4_pack(y[at])
    assert torch.equal(c2[at], wc) and torch.equal(s2[at], ws)


def test_norm_and_its_gradient(dev):
    rows, h = 540_000, 8192
    print("norm", flush=True)
    assert rows * h > GIB4  # the 8-bit rows too
    at = _at(dev, rows, h)
    x, res, w = _rand(dev, rows, h), _rand(dev, rows, h, seed=1), (1 + 0.2 * _rand(dev, h, seed=2).float()).bfloat16()
    far = mtb.rmsnorm_mxfp8(x, w, res)
    alone = mtb.rmsnorm_mxfp8(x[at], w, res[at])
    for a, b in zip(far, alone):
        assert torch.equal(a[at], b)
    data, scales, hh, rstd = far
    del x, data, scales, far
    dx, dw = mtb.drmsnorm(res, hh, w, rstd)
    assert torch.equal(dx[at], mtb.drmsnorm(res[at].contiguous(), hh[at].contiguous(), w, rstd[at])[0])
    # dweight from the far rows alone
    res.zero_()
    res[at] = _rand(dev, len(at), h, seed=3)
    _, dw = mtb.drmsnorm(res, hh, w, rstd)
    t = res[at].double() * hh[at].double() * rstd[at].double()[:, None]
    assert bool(((dw.double() - t.sum(0)).abs() <= (len(at) + 3) * U * t.abs().sum(0)).all())
