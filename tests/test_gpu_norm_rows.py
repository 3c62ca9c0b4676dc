"""The norm's row statistics at bars that do not grow with the row, so that one value
left out of a wide row's sum shows.

With u = 2^-24.  rstd: eight squares are added in FP32 (eight roundings of positive terms,
8 u of their sum), the eights, the mean, eps, the root and the quotient in FP64; halved by
the root and rounded once to FP32: (8 / 2 + 1) u, second orders within 0.01 u.  Where every eight's sum is a
whole number below 2^24 nothing is rounded before the last step, and rstd is the FP32
number nearest to the exact one.

The gradient's mean(g h): a thread adds at most 32 terms in FP32, a wave's 64 threads in 6
steps, at most 8 waves one after the other: at most 46 roundings, one more in g's own
product, 4 in the factors 1 / H, 1 / H's own, r and r: 52 u of mean |g h| r^2, second orders
within one more."""

import numpy as np
import pytest
import torch

import moe_token_block_amd as mtb
from oracle import formats as F
from oracle import expert, products

from gpu_util import require_gpu, bf16_dev, host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# every number of threads a row and of chunks a thread, whole and cut
WIDTHS = [32, 96, 512, 544, 1024, 1056, 2048, 2080, 4096, 4128, 7168, 8192, 8224, 12000, 16384]


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _bits(x):
    return F.f32_to_bf16(np.asarray(x, dtype=np.float32))


def _places(h):
    """The first and last value, and one of every wave's 512 neighbours."""
    at = {0, 7, h // 2, h - 8, h - 1}
    at.update(min(o + 37, h - 1) for o in range(0, h, 512))
    return sorted(p for p in at if p >= 0)


def _one_place(h, small):
    """A row for each place: `small` everywhere but for one value that carries the sum."""
    places = _places(h)
    x = np.full((len(places), h), small)
    x[np.arange(len(places)), places] = 8.0 + np.arange(len(places)) / 16.0
    return x


def _rstd(dev, bits, eps):
    w = torch.ones(bits.shape[1], dtype=torch.bfloat16, device=dev)
    return host(mtb.rmsnorm_mxfp8(bf16_dev(bits, dev), w, eps=eps)[3])


@pytest.mark.parametrize("h", WIDTHS)
def test_rstd(dev, h):
    print(f"rstd {h}", flush=True)
    rng = np.random.default_rng(h)
    x = np.concatenate([rng.standard_normal((40, h)) * np.exp(rng.standard_normal((40, 1))), _one_place(h, 2.0 ** -6),
                        _one_place(h, 0.0)])
    bits = _bits(x)
    want, _ = products.rmsnorm(expert.f64(bits), np.ones(h), 1e-6)
    off = np.abs(_rstd(dev, bits, 1e-6) - want) / want
    assert off.max() <= 5.01 * U, (int(off.argmax()), off.max() / U)


@pytest.mark.parametrize("h", WIDTHS)
def test_rstd_is_the_nearest_where_the_eights_are_exact(dev, h):
    """Whole numbers up to 255: an eight's squares add up to less than 2^19, a wide row's to more than 2^24."""
    rng = np.random.default_rng(h + 1)
    x = rng.integers(-255, 256, (64, h)).astype(np.float64)
    eps = np.float32(1e-6)
    mean = (x * x).sum(1).astype(np.longdouble) / h + np.longdouble(eps)
    want = 1 / np.sqrt(mean)
    got = _rstd(dev, _bits(x), float(eps))
    near = want.astype(np.float32)
    # a few FP64 roundings ahead of the last one may decide a tie: 2^-51 of the value around it
    half = np.spacing(near).astype(np.longdouble) / 2
    sure = np.abs(np.abs(want - near.astype(np.longdouble)) - half) > want * np.longdouble(2.0) ** -51
    assert sure.sum() >= 60 and np.array_equal(got[sure], near[sure])


def _gradient(dev, dy, x, w, eps=1e-6):
    rstd = (1 / np.sqrt((expert.f64(x) ** 2).mean(axis=1) + eps)).astype(np.float32)
    dx, _ = mtb.drmsnorm(*(bf16_dev(v, dev) for v in (dy, x, w)), torch.from_numpy(rstd).to(dev))
    y, f, ww = expert.f64(dy), expert.f64(x), expert.f64(w)
    want, _ = products.drmsnorm(y, f, ww, rstd.astype(np.float64), None)
    g, r = y * ww, rstd.astype(np.float64)[:, None]
    kmag = np.abs(g * f).mean(1, keepdims=True) * r * r
    # and, behind the mean: g's product, the product with h, their difference and the product with r
    slack = r * (53 * U * np.abs(f) * kmag + 4 * U * (np.abs(g) + np.abs(f) * kmag))
    off = np.abs(dx.double().cpu().numpy() - want) - (slack + 2.0 ** -8 * (np.abs(want) + slack) + 2.0 ** -134)
    assert not (off > 0).any(), np.unravel_index(off.argmax(), off.shape)


@pytest.mark.parametrize("rows", [3, 6])  # one workgroup for all rows; one for each
@pytest.mark.parametrize("h", WIDTHS)
def test_gradient_where_the_mean_counts(dev, h, rows):
    """dy along h: what is left of dx is small beside each of its two parts, so that a term
    missing from the mean shows."""
    print(f"gradient {h} {rows}", flush=True)
    rng = np.random.default_rng(h + rows)
    x = _bits(rng.standard_normal((rows, h)))
    ones = _bits(np.ones(h))
    _gradient(dev, x, x, ones)
    _gradient(dev, _bits(expert.f64(x) * 0.75), x, _bits(np.full(h, 1.5)))
    _gradient(dev, _bits(expert.f64(x) + 2.0 ** -9 * rng.standard_normal((rows, h))), x, ones)


@pytest.mark.parametrize("h", WIDTHS)
def test_gradient_of_one_place(dev, h):
    """One product carries the mean: every other dx is that product's."""
    rng = np.random.default_rng(h + 2)
    places = _places(h)
    n = len(places)
    x = rng.standard_normal((n, h))
    dy = np.zeros((n, h))
    dy[np.arange(n), places] = 1.0 + np.arange(n) / 32.0
    x[np.arange(n), places] = 8.0
    for lo in range(0, n, 4):  # up to four rows: one workgroup
        _gradient(dev, _bits(dy[lo:lo + 4]), _bits(x[lo:lo + 4]), _bits(1 + 0.2 * rng.standard_normal(h)))
    _gradient(dev, _bits(dy), _bits(x), _bits(1 + 0.2 * rng.standard_normal(h)))
