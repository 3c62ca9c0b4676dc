"""MXFP8 and MXFP4 rows times MXFP4 weights where the terms cancel, so that no final rounding hides
what the sum loses.

Every value is chosen so that each term is a multiple of 2^-7 and the terms' magnitudes
add up to less than 2^17 (MXFP4 rows: of 2^-2, less than 2^22): FP32 holds any partial sum,
in any order, and the result has to be the BF16 nearest to the exact sum (in float64,
which holds it too), bit for bit."""

import pytest
import torch

import moe_token_block_amd as mtb
from oracle import formats as F

from gpu_util import require_gpu
from test_gpu_products_large import _plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _e4m3(v):
    """Bytes of values that E4M3 holds."""
    table = torch.from_numpy(F.e4m3_decode(torch.arange(127, dtype=torch.uint8).numpy())).to(v.device)
    at = torch.searchsorted(table, v.abs())
    assert torch.equal(table[at], v.abs())
    return at.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 7)


def _terms(g, r, n, k):
    """Rows [r, k] with pairs of +-448 in up to 16 groups of eight neighbours and values of
    multiples of 1/64 below 1/4 beside them; weight codes [n, k] that are 6 where the pairs
    are: 16 * 2 * 2688 + k * 6 / 4 < 2^17 for k < 2^14."""
    dev = g.device
    x = torch.randint(-15, 16, (r, k), generator=g, device=dev).double() / 64
    codes = torch.randint(0, 16, (n, k), generator=g, device=dev).to(torch.uint8)
    for eight in torch.randperm(k // 8, generator=g, device=dev)[:16].tolist():
        i, j = (8 * eight + torch.randperm(8, generator=g, device=dev)[:2]).tolist()
        x[:, i] = 448.0 * (2 * torch.randint(0, 2, (r,), generator=g, device=dev) - 1)
        x[:, j] = -x[:, i]
        codes[:, i] = codes[:, j] = 7
    return x, codes


def _values(codes):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=codes.device)
    return torch.cat([grid, -grid])[codes.int()]


# counts, hidden, width: few rows; a long sum left to few tiles; two groups of waves a tile;
# one; two column tiles that are cut; large tiles, whole steps and a last one that is cut
CASES = [([5, 16, 1], 32, 40), ([9, 0, 3], 1056, 33), ([120, 3, 400], 4128, 130), ([380, 420, 400], 1632, 500),
         ([70] * 24, 288, 1100), ([200, 260, 512, 700], 864, 4101), ([200, 190, 210, 250] * 6, 416, 16380)]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_terms_that_cancel(dev, case):
    counts, k, n = CASES[case]
    print(f"case {case}: {CASES[case]}", flush=True)
    g = torch.Generator(device=dev).manual_seed(case)
    plan, offsets, used = _plan(counts, 16, dev)
    r, e = plan["r_cap"], len(counts)
    data = torch.zeros((r, k), dtype=torch.uint8, device=dev)
    wc = torch.empty((e, n, k // 2), dtype=torch.uint8, device=dev)
    want = torch.zeros((r, n), dtype=torch.bfloat16, device=dev)
    for i, (c, o) in enumerate(zip(counts, offsets)):
        x, codes = _terms(g, c, n, k)
        data[o:o + c] = _e4m3(x)
        wc[i] = codes[:, ::2] | (codes[:, 1::2] << 4)
        want[o:o + c] = (x @ _values(codes).T.contiguous()).float().bfloat16()  # exact before the last step
    for a, b in ((127, 127), (7, 247), (247, 7)):  # scales 2^-120 and 2^120 of the two sides leave the terms as they are
        s = torch.full((r, k // 32), a, dtype=torch.uint8, device=dev)
        ws = torch.full((e, n, k // 32), b, dtype=torch.uint8, device=dev)
        got = mtb.ep_mxfp4_grouped_gemm(data, s, wc, ws, plan)
        off = (got != want).nonzero()
        assert not len(off), (a, b, len(off), got.numel(), off[0].tolist(), got[tuple(off[0])].item(), want[tuple(off[0])].item())


@pytest.mark.parametrize("case", range(len(CASES)))
def test_four_bit_terms_that_cancel(dev, case):
    """Up to 16 blocks of 32 at 2^9 of the others' scale, each with a pair of +-6 times 6 and else
    0.5 times 0.5 or 1: 16 * (72 + 15) * 2^9 + k * 36 < 2^22 for k < 2^16."""
    counts, k, n = CASES[case]
    print(f"case {case}: {CASES[case]}", flush=True)
    g = torch.Generator(device=dev).manual_seed(case)
    plan, offsets, used = _plan(counts, 16, dev)
    r, e = plan["r_cap"], len(counts)
    ints = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device=dev).to(torch.uint8)  # noqa: E731
    data = torch.zeros((r, k // 2), dtype=torch.uint8, device=dev)
    s = torch.full((r, k // 32), 127, dtype=torch.uint8, device=dev)
    wc = torch.empty((e, n, k // 2), dtype=torch.uint8, device=dev)
    want = torch.zeros((r, n), dtype=torch.bfloat16, device=dev)
    pack = lambda c: c[:, ::2] | (c[:, 1::2] << 4)  # noqa: E731
    for i, (c, o) in enumerate(zip(counts, offsets)):
        x, codes = ints(0, 16, c, k), ints(0, 16, n, k)
        scales = torch.full((c, k // 32), 127, dtype=torch.uint8, device=dev)
        for b in torch.randperm(k // 32, generator=g, device=dev)[:16].tolist():
            at = slice(32 * b, 32 * b + 32)
            x[:, at], codes[:, at] = 1 + 8 * ints(0, 2, c, 32), 1 + ints(0, 2, n, 32)
            p, q = (32 * b + torch.randperm(32, generator=g, device=dev)[:2]).tolist()
            x[:, p] = 7 + 8 * ints(0, 2, c)
            x[:, q] = x[:, p] ^ 8
            codes[:, p] = codes[:, q] = 7
            scales[:, b] = 127 + 9
        data[o:o + c], wc[i], s[o:o + c] = pack(x), pack(codes), scales
        a = _values(x) * (scales.double() - 127).exp2().repeat_interleave(32, 1)
        want[o:o + c] = (a @ _values(codes).T.contiguous()).float().bfloat16()
    for a, b in ((0, 0), (-120, 118), (110, -110)):
        ws = torch.full((e, n, k // 32), 127 + b, dtype=torch.uint8, device=dev)
        got = mtb.ep_mxfp4_grouped_gemm(data, (s.int() + a).to(torch.uint8), wc, ws, plan)
        exact = (want.double() * 2.0 ** (a + b)).bfloat16()  # a power of two: no rounding
        off = (got != exact).nonzero()
        assert not len(off), (a, b, len(off), got.numel(), off[0].tolist(), got[tuple(off[0])].item(), exact[tuple(off[0])].item())


@pytest.mark.parametrize("counts,k,n", [([5, 16, 1], 96, 40), ([380, 420, 400], 160, 500), ([70] * 24, 96, 1100),
                                        ([200] * 24, 96, 16384)])
def test_a_nan_byte_reaches_its_row_alone(dev, counts, k, n):
    """0x7F and 0xFF are E4M3's NaN: their row's results are NaN, every other row's as without it."""
    g = torch.Generator(device=dev).manual_seed(n)
    plan, offsets, used = _plan(counts, 16, dev)
    r, e = plan["r_cap"], len(counts)
    rand = lambda *shape: torch.randint(0, 256, shape, generator=g, device=dev).to(torch.uint8)  # noqa: E731
    data, wc = rand(r, k), rand(e, n, k // 2)
    data[(data & 127) == 127] = 0
    s = torch.full((r, k // 32), 127, dtype=torch.uint8, device=dev)
    ws = torch.full((e, n, k // 32), 127, dtype=torch.uint8, device=dev)
    clean = mtb.ep_mxfp4_grouped_gemm(data, s, wc, ws, plan)
    at = [int(offsets[0]) + 2, int(offsets[1]) + counts[1] - 1]
    data[at[0], k - 1], data[at[1], 7] = 0x7F, 0xFF
    got = mtb.ep_mxfp4_grouped_gemm(data, s, wc, ws, plan)
    assert bool(got[at].isnan().all())
    rest = torch.ones(r, dtype=torch.bool, device=dev)
    rest[at] = False
    assert torch.equal(got[rest].view(torch.int16), clean[rest].view(torch.int16))
