"""The grouped BF16 products with values at the ends of their range, and the weights'
gradient by its large tiles where they are too many for one XCD.

With u = 2^-24: products of BF16 numbers, subnormal ones among them, are exact in FP32
wherever FP32 is normal; a sum of n terms is within (n + 1) u of the sum of the terms'
magnitudes, and each step below FP32's normal range loses at most 2^-149.  The matrix unit
takes a BF16 number below the normal range with the exponent -126 and leading zeros (with
rows of such numbers alone, bits of a sum that FP32 would hold are cut at 2^-24 of that
exponent's product: up to 2^7 of the terms' own), so it counts among the magnitudes
as 2^-126.  An infinity or a NaN of an entry reaches what it is a term of and nothing else."""

import pytest
import torch

import moe_token_block_amd as mtb

from gpu_util import require_gpu
from test_gpu_products_large import _plan, _near, _rand

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


# counts, hidden, width: more than 32 tiles of 256 x 256 an expert, 256 and more in all;
# whole tiles, odd widths, a number of tiles that eight XCDs do not share evenly
WGRAD = [([0, 1, 64, 65, 700], 2048, 1792), ([130, 63, 2, 0, 300], 1701, 1999), ([40] * 7, 1700, 1530), ([257] * 2, 5000, 3333)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", range(len(WGRAD)))
def test_weights_gradient_by_many_large_tiles(dev, case, dtype):
    counts, k, n = WGRAD[case]
    per = -(-n // 256) * -(-k // 256)
    assert per > 32 and per * len(counts) >= 256
    print(f"case {case}: {WGRAD[case]} {dtype}", flush=True)
    g = torch.Generator(device=dev).manual_seed(case)
    plan, offsets, used = _plan(counts, 16, dev, 30)
    x, d = _rand(g, plan["r_cap"], k), _rand(g, plan["r_cap"], n)
    x[~used], d[~used] = float("nan"), float("nan")
    out = torch.full((len(counts), n, k), float("nan"), dtype=dtype, device=dev)
    got = mtb.ep_bf16_grouped_wgrad(d, x, plan, out=out)
    for i, (c, o) in enumerate(zip(counts, offsets)):
        a, b = d[o:o + c].double().T.contiguous(), x[o:o + c].double()
        _near(got[i], a @ b, (c + 1) * U * (a.abs() @ b.abs()), ("wgrad", i), U if dtype is torch.float32 else 2.0 ** -8)


# one for each kernel of the product, of the rows' gradient and of the weights' gradient:
# few rows 16 and 32 at a time; small tiles of two groups of waves and of one; large tiles
SHAPES = [([9] * 40, 130, 72), ([20] * 40, 200, 1100), ([380, 420, 400], 264, 500), ([70] * 24, 136, 1100),
          ([200, 260, 512, 700], 200, 4101), ([200, 260, 512, 700], 4101, 200), ([40] * 7, 1700, 1530)]


def _all(plan, x, d, w):
    return (mtb.ep_bf16_grouped_gemm(x, w, plan), mtb.ep_bf16_grouped_dgrad(d, w, plan), mtb.ep_bf16_grouped_wgrad(d, x, plan),
            mtb.ep_bf16_grouped_wgrad(d, x, plan, dtype=torch.float32))


def _size(v):
    return torch.where(v == 0, 0.0, v.abs().clamp(min=2.0 ** -126))


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_subnormal_and_far_values(dev, case):
    """Rows below BF16's normal range times large weights and gradients; products that are
    themselves below FP32's normal range; large times small."""
    counts, k, n = SHAPES[case]
    print(f"case {case}: {SHAPES[case]}", flush=True)
    g = torch.Generator(device=dev).manual_seed(case)
    plan, offsets, used = _plan(counts, 16, dev)
    r, e = plan["r_cap"], len(counts)
    # powers of two for the scales of (rows, the other two)
    for a, b in ((-128, 100), (-130, 20), (100, -128), (-70, -62)):
        x, d, w = _rand(g, r, k), _rand(g, r, n), _rand(g, e, n, k)
        x, d, w = (x.double() * 2.0 ** a).bfloat16(), (d.double() * 2.0 ** b).bfloat16(), (w.double() * 2.0 ** b).bfloat16()
        x2 = (d.double() * 2.0 ** (a - b)).bfloat16()  # the rows' gradient: of dout as small as x
        out, dx, dw, dw32 = _all(plan, x, d, w)
        dx = mtb.ep_bf16_grouped_dgrad(x2, w, plan)
        for i, (c, o) in enumerate(zip(counts, offsets)):
            at = slice(o, o + c)
            for got, p, q, terms, step in ((out[at], x[at].double(), w[i].double().T.contiguous(), k, 2.0 ** -8),
                                           (dx[at], x2[at].double(), w[i].double(), n, 2.0 ** -8),
                                           (dw[i], d[at].double().T.contiguous(), x[at].double(), c, 2.0 ** -8),
                                           (dw32[i], d[at].double().T.contiguous(), x[at].double(), c, U)):
                want, mag = p @ q, _size(p) @ _size(q)
                _near(got, want, (terms + 1) * U * mag + 2 * terms * 2.0 ** -149, (a, b, i, terms), step)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_an_infinity_or_a_nan_of_an_entry(dev, case, value):
    counts, k, n = SHAPES[case]
    print(f"case {case}: {SHAPES[case]} {value}", flush=True)
    g = torch.Generator(device=dev).manual_seed(case)
    plan, offsets, used = _plan(counts, 16, dev)
    r, e = plan["r_cap"], len(counts)
    x, d, w = _rand(g, r, k), _rand(g, r, n), _rand(g, e, n, k)
    clean = _all(plan, x, d, w)

    def same(got, want, what):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), what

    def like(got, factor, what):
        """got: value times each factor; a factor of 0 makes a NaN."""
        want = factor.double() * value
        assert torch.equal(got.double().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0)), what

    last = e - 1
    places = [(0, int(offsets[0]), 0, 0), (last, int(offsets[last]) + counts[last] - 1, k - 1, n - 1)]
    for i, row, kk, nn in places:  # one at the front of everything, one at the end
        at = slice(int(offsets[i]), int(offsets[i]) + counts[i])
        bad = x.clone()
        bad[row, kk] = value
        out, _, dw, dw32 = _all(plan, bad, d, w)
        like(out[row], w[i, :, kk], "gemm by a row")
        out[row] = clean[0][row]
        same(out, clean[0], "gemm, other rows")
        for got, was in ((dw, clean[2]), (dw32, clean[3])):
            like(got[i, :, kk], d[row], "wgrad by a row")
            got[i, :, kk] = was[i, :, kk]
            same(got, was, "wgrad, other columns")
        bad = d.clone()
        bad[row, nn] = value
        _, dx, dw, dw32 = _all(plan, x, bad, w)
        like(dx[row], w[i, nn], "dgrad by a row")
        dx[row] = clean[1][row]
        same(dx, clean[1], "dgrad, other rows")
        for got, was in ((dw, clean[2]), (dw32, clean[3])):
            like(got[i, nn], x[row], "wgrad by dout")
            got[i, nn] = was[i, nn]
            same(got, was, "wgrad, other rows")
        bad = w.clone()
        bad[i, nn, kk] = value
        out, dx, _, _ = _all(plan, x, d, bad)
        like(out[at, nn], x[at, kk], "gemm by a weight")
        like(dx[at, kk], d[at, nn], "dgrad by a weight")
        out[at, nn], dx[at, kk] = clean[0][at, nn], clean[1][at, kk]
        same(out, clean[0], "gemm, other experts and columns")
        same(dx, clean[1], "dgrad, other experts and columns")


def _cancel(g, m, terms, cols):
    """Factors [m, terms] and [terms, cols] whose products are multiples of 2^-11, at most 225 *
    2^-11 but for one pair of +-2048 a result: less than 2^13 in all for up to 30000 terms,
    so that FP32 holds any partial sum in any order."""
    a = torch.randint(-15, 16, (m, terms), generator=g, device=g.device).double() / 64
    b = torch.randint(-15, 16, (terms, cols), generator=g, device=g.device).double() / 32
    if terms > 1:
        i, j = torch.randperm(terms, generator=g, device=g.device)[:2].tolist()
        a[:, i] = 32.0 * (2 * torch.randint(0, 2, (m,), generator=g, device=g.device) - 1)
        a[:, j] = -a[:, i]
        b[i] = b[j] = 64.0
    return a, b


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_terms_that_cancel(dev, case):
    """The results are the exact sums, rounded once where they are BF16, bit for bit."""
    counts, k, n = SHAPES[case]
    print(f"case {case}: {SHAPES[case]}", flush=True)
    g = torch.Generator(device=dev).manual_seed(case)
    plan, offsets, used = _plan(counts, 16, dev)
    r, e = plan["r_cap"], len(counts)
    zeros = lambda *s: torch.zeros(s, dtype=torch.float64, device=dev)  # noqa: E731
    spans = [(i, slice(int(o), int(o) + c)) for i, (c, o) in enumerate(zip(counts, offsets))]

    def equal(got, want, what):
        want = want.float().to(got.dtype)
        off = (got != want).nonzero()
        assert not len(off), (what, len(off), off[0].tolist(), got[tuple(off[0])].item(), want[tuple(off[0])].item())

    x, w, want = zeros(r, k), zeros(e, n, k), zeros(r, n)
    for i, at in spans:
        x[at], q = _cancel(g, counts[i], k, n)
        w[i], want[at] = q.T, x[at] @ q
    equal(mtb.ep_bf16_grouped_gemm(x.bfloat16(), w.bfloat16(), plan), want, "gemm")
    d, want = zeros(r, n), zeros(r, k)
    for i, at in spans:
        d[at], w[i] = _cancel(g, counts[i], n, k)
        want[at] = d[at] @ w[i]
    equal(mtb.ep_bf16_grouped_dgrad(d.bfloat16(), w.bfloat16(), plan), want, "dgrad")
    want = zeros(e, n, k)
    for i, at in spans:
        p, x[at] = _cancel(g, n, counts[i], k)
        d[at], want[i] = p.T, p @ x[at]
    for dtype in (torch.bfloat16, torch.float32):
        equal(mtb.ep_bf16_grouped_wgrad(d.bfloat16(), x.bfloat16(), plan, dtype=dtype), want, "wgrad")
