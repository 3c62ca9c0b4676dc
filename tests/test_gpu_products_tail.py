"""Products whose plan has many rows behind the last expert's, by the kernels for few rows
with one and with several workgroups beside each other: every row there is cleared, every
result above it is right.  Bars as for the other sizes, with u = 2^-24: (n + 1) u of the
sum of the terms' magnitudes before the rounding."""

import pytest
import torch

import moe_token_block_amd as mtb

from gpu_util import require_gpu
from test_gpu_products_large import _check_rows, _plan, _rand

pytestmark = pytest.mark.gpu

# counts, hidden, width, rows behind: one workgroup an expert and stretch, several, more than stretches
CASES = [([3] * 70, 96, 1100, 5000), ([40, 9], 72, 16, 70_000), ([900, 700], 64, 24, 1000), ([500, 0, 300], 2080, 40, 3001),
         ([20] * 3, 96, 100, 257), ([0, 0], 96, 40, 100_000)]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_rows_behind_the_last_expert(case):
    dev = require_gpu()
    counts, k, n, extra = CASES[case]
    print(f"case {case}: {CASES[case]}", flush=True)
    g = torch.Generator(device=dev).manual_seed(case)
    plan, offsets, used = _plan(counts, 16, dev, extra)
    r, e = plan["r_cap"], len(counts)
    x, d, w = _rand(g, r, k), _rand(g, r, n), _rand(g, e, n, k)
    x[~used], d[~used] = float("nan"), float("nan")
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device=dev)  # noqa: E731
    _check_rows(mtb.ep_bf16_grouped_gemm(x, w, plan, out=nan(r, n)), lambda at: x[at].double(),
                lambda i: w[i].double().T.contiguous(), counts, offsets, used, k, 0.0, "gemm")
    _check_rows(mtb.ep_bf16_grouped_dgrad(d, w, plan, out=nan(r, k)), lambda at: d[at].double(), lambda i: w[i].double(),
                counts, offsets, used, n, 0.0, "dgrad")
    if k % 32:
        return
    wc, ws = (v.view(e, n, -1) for v in mtb.ep_mxfp4_pack(w.view(-1, k)))
    rows = x.nan_to_num(nan=0.0)
    for (q, s), decode in ((mtb.ep_mxfp4_pack(rows), mtb.ep_mxfp4_unpack), (mtb.ep_mxfp8_pack(rows)[:2], mtb.ep_mxfp8_unpack)):
        values = decode(q, s)
        s[~used] = 255
        _check_rows(mtb.ep_mxfp4_grouped_gemm(q, s, wc, ws, plan, out=nan(r, n)), lambda at: values[at].double(),
                    lambda i: mtb.ep_mxfp4_unpack(wc[i], ws[i]).double().T.contiguous(), counts, offsets, used, k, 0.0, "mx")
