"""The grouped products' tile kernels as a program uses them: operands and results at any
address, a captured graph whose plan changes between replays, two calls at once on two
streams, as many experts as the calls take.  Compared with the same call on aligned
copies, eager and alone, bit for bit (no call's result depends on any of these); many
experts against float64 at the bars of the small sizes."""

import pytest
import torch

import moe_token_block_amd as mtb

from gpu_util import require_gpu
from test_gpu_products_large import _check_rows, _near, _plan, _rand

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# small tiles of two groups of waves and of one, large tiles, shares of the weights' gradient
CASES = [([380, 420, 400], 1632, 500), ([70] * 24, 288, 1100), ([200, 260, 512, 700], 864, 4101), ([3000, 2500], 160, 72),
         ([200] * 24, 96, 16384)]


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _inputs(dev, case):
    counts, k, n = CASES[case]
    print(f"case {case}: {CASES[case]}", flush=True)
    g = torch.Generator(device=dev).manual_seed(case)
    plan, offsets, used = _plan(counts, 16, dev)
    r, e = plan["r_cap"], len(counts)
    x, d, w = _rand(g, r, k), _rand(g, r, n), _rand(g, e, n, k)
    wc, ws = (v.view(e, n, -1) for v in mtb.ep_mxfp4_pack(w.view(-1, k)))
    c4, s4 = mtb.ep_mxfp4_pack(x)
    c8, s8, _ = mtb.ep_mxfp8_pack(x)
    return plan, dict(x=x, d=d, w=w, wc=wc, ws=ws, c4=c4, s4=s4, c8=c8, s8=s8)


CALLS = [("gemm", lambda v, p, o=None: mtb.ep_bf16_grouped_gemm(v["x"], v["w"], p, out=o)),
         ("dgrad", lambda v, p, o=None: mtb.ep_bf16_grouped_dgrad(v["d"], v["w"], p, out=o)),
         ("wgrad", lambda v, p, o=None: mtb.ep_bf16_grouped_wgrad(v["d"], v["x"], p, out=o)),
         ("wgrad32", lambda v, p, o=None: mtb.ep_bf16_grouped_wgrad(v["d"], v["x"], p, out=o, dtype=torch.float32)),
         ("mx4", lambda v, p, o=None: mtb.ep_mxfp4_grouped_gemm(v["c4"], v["s4"], v["wc"], v["ws"], p, out=o)),
         ("mx8", lambda v, p, o=None: mtb.ep_mxfp4_grouped_gemm(v["c8"], v["s8"], v["wc"], v["ws"], p, out=o))]


def _same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def _shifted(t, by):
    """A copy that begins `by` elements behind an aligned address, 64 elements of 7 on its other side."""
    b = torch.full((t.numel() + by + 64,), 7, dtype=t.dtype, device=t.device)
    b[by:by + t.numel()] = t.reshape(-1)
    return b[by:by + t.numel()].view(t.shape), b


@pytest.mark.parametrize("case", range(len(CASES)))
def test_any_address(dev, case):
    plan, v = _inputs(dev, case)
    want = [call(v, plan) for _, call in CALLS]
    for by in (1, 3):
        odd = {k: _shifted(t, by)[0] for k, t in v.items()}
        for (name, call), was in zip(CALLS, want):
            out, all_of_it = _shifted(torch.full_like(was, float("nan")), by)
            call(odd, plan, out)
            assert _same(out, was), (name, by)
            assert bool((all_of_it[:by] == 7).all()) and bool((all_of_it[by + was.numel():] == 7).all()), (name, by)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_replays_with_other_plans(dev, case):
    plan, v = _inputs(dev, case)
    outs = [torch.empty_like(call(v, plan)) for _, call in CALLS]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for (_, call), o in zip(CALLS, outs):
            call(v, plan, o)
    counts, offsets = plan["counts"].clone(), plan["offsets"].clone()
    e, room = len(counts), int(offsets[-1]) // len(counts) // 16 * 16
    even = torch.arange(e + 1, dtype=torch.int32, device=dev) * room
    for c, o in ((counts, offsets), (counts // 2, offsets), (torch.full_like(counts, room), even),
                 (torch.arange(e, dtype=torch.int32, device=dev) % 3 * (room // 2), even), (counts, offsets)):
        plan["counts"].copy_(c)
        plan["offsets"].copy_(o)
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for (name, call), got in zip(CALLS, outs):
            assert _same(got, call(v, plan, torch.full_like(got, float("nan")))), name


def test_two_calls_at_once(dev):
    """Different calls, and a call and itself, side by side on two streams."""
    sets = [_inputs(dev, case) for case in (0, 2, 3)]
    want = [[call(v, plan) for _, call in CALLS] for plan, v in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = [[], []]
    for turn in range(2):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for j in range(len(sets)):
                    plan, v = sets[(j + i * turn) % len(sets)]
                    got[i].append([call(v, plan) for _, call in CALLS])
    torch.cuda.synchronize()
    for i in range(2):
        for turn in range(2):
            for j in range(len(sets)):
                at = (j + i * turn) % len(sets)
                for (name, _), a, b in zip(CALLS, got[i][turn * len(sets) + j], want[at]):
                    assert _same(a, b), (name, i, turn, j)


# most experts without a row, all with some, one with nearly all; the rows behind the last
MANY = [([0] * 1000 + [5, 0, 17, 300] * 6, 96, 40, 300), ([30, 1, 0, 64] * 256, 96, 136, 0), ([3] * 63 + [6000] + [3] * 960, 64, 72, 17),
        ([7, 0] * 512, 224, 33, 5000)]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_experts(dev, case):
    counts, k, n, extra = MANY[case]
    assert len(counts) == 1024
    print(f"case {case}", flush=True)
    g = torch.Generator(device=dev).manual_seed(case)
    plan, offsets, used = _plan(counts, 16, dev, extra)
    r, e = plan["r_cap"], len(counts)
    x, d, w = _rand(g, r, k), _rand(g, r, n), _rand(g, e, n, k)
    wc, ws = (v.view(e, n, -1) for v in mtb.ep_mxfp4_pack(w.view(-1, k)))
    (c4, s4), (c8, s8, _) = mtb.ep_mxfp4_pack(x), mtb.ep_mxfp8_pack(x)
    x4, x8 = mtb.ep_mxfp4_unpack(c4, s4), mtb.ep_mxfp8_unpack(c8, s8)
    w4 = mtb.ep_mxfp4_unpack(wc.view(e * n, -1), ws.view(e * n, -1)).view(e, n, k)
    s4[~used], s8[~used], x[~used], d[~used] = 255, 255, float("nan"), float("nan")
    out = [mtb.ep_bf16_grouped_gemm(x, w, plan), mtb.ep_bf16_grouped_dgrad(d, w, plan),
           mtb.ep_mxfp4_grouped_gemm(c4, s4, wc, ws, plan), mtb.ep_mxfp4_grouped_gemm(c8, s8, wc, ws, plan)]
    dw = mtb.ep_bf16_grouped_wgrad(d, x, plan, dtype=torch.float32)
    some = [i for i in (0, 1, 62, 63, 64, 65, 127, 128, 500, 511, 512, 999, 1000, 1002, 1003, 1020, 1022, 1023) if counts[i]]
    c, o = [counts[i] if i in some else 0 for i in range(e)], offsets
    for got, rows, weight, terms, what in ((out[0], x, lambda i: w[i].double().T.contiguous(), k, "gemm"),
                                           (out[1], d, lambda i: w[i].double(), n, "dgrad"),
                                           (out[2], x4, lambda i: w4[i].double().T.contiguous(), k, "mx4"),
                                           (out[3], x8, lambda i: w4[i].double().T.contiguous(), k, "mx8")):
        _check_rows(got, lambda at: rows[at].double(), weight, c, o, used, terms, 0.0, what)
    empty = torch.tensor([m == 0 for m in counts], device=dev)
    assert not bool(dw[empty].any())
    for i in some:
        a, b = d[o[i]:o[i] + counts[i]].double().T.contiguous(), x[o[i]:o[i] + counts[i]].double()
        _near(dw[i], a @ b, (counts[i] + 1) * U * (a.abs() @ b.abs()), ("wgrad", i), U)
