"""The grouped products at sizes where the rules pick their other kernels: large tiles,
small ones with one group of waves and with two, the kernels for few rows with one and
with several workgroups an expert, a weight gradient in shares; loads that are very
uneven, every expert's count at and around the tiles' edges.

Compared on the GPU with torch in 64 bits (sampled rows where all would take long);
bars as for the small sizes, with u = 2^-24: (n + 1) u of the sum of the terms'
magnitudes before the rounding, 2^-10 of it more for MXFP8 rows."""

import numpy as np
import pytest
import torch

import moe_token_block_amd as mtb

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _plan(counts, align, dev, extra=0):
    """The plan of experts with these counts, its unused rows and `extra` more behind."""
    counts = np.asarray(counts)
    offsets = np.concatenate([[0], np.cumsum((counts + align - 1) // align * align)])
    r_cap = int(offsets[-1]) + extra
    used = np.zeros(r_cap, dtype=bool)
    for c, o in zip(counts, offsets):
        used[o:o + c] = True
    dst = np.nonzero(used)[0].astype(np.int32).reshape(-1, 1)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    return dict(counts=i32(counts), offsets=i32(offsets), dst_row=i32(dst), src_row=i32(np.where(used, 0, -1)),
                r_cap=r_cap, num_experts=len(counts), alignment=align), offsets, torch.from_numpy(used).to(dev)


def _near(got, want, slack, what, step=2.0 ** -8):
    bad = ~((got.double() - want).abs() <= slack + step * (want.abs() + slack) + 2.0 ** -134)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.numel(), [int(b[0]) for b in bad.nonzero(as_tuple=True)])


def _check_rows(got, x, w, counts, offsets, used, terms, more, what):
    """got[g] = w[e] x[g] (w(e): 64-bit [terms, columns]), zeros elsewhere."""
    assert not bool(got[~used].any()), what
    for e, (c, o) in enumerate(zip(counts, offsets)):
        if c == 0:
            continue
        at = torch.arange(o, o + c, device=got.device)
        if c > 64:  # both ends, the tiles' edges and some between
            at = at[torch.unique(torch.cat([torch.arange(0, 12), torch.arange(c - 12, c), torch.arange(124, 132).clamp(max=c - 1),
                                            torch.arange(252, 260).clamp(max=c - 1), torch.arange(0, c, c // 16)]))]
        a, b = x(at), w(e)
        _near(got[at], a @ b, ((terms + 1) * U + more) * (a.abs() @ b.abs()), (what, e))


def _rand(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device=g.device, dtype=torch.float32).mul_(scale).bfloat16()


# counts, hidden, width, alignment, rows behind
EDGES = [1, 0, 15, 16, 17, 127, 128, 129, 255, 256, 257, 300]
CASES = [
    (EDGES, 200, 264, 16, 40),                               # blocks of 32 rows, several an expert
    (EDGES, 192, 3000, 1, 0),                                # small tiles, offsets of any kind
    ([900] + [0] * 14 + [3], 1608, 640, 16, 300),            # one expert has nearly all
    ([380, 420, 400], 1600, 500, 16, 0),                     # fewer tiles than CUs: two groups of waves
    ([380, 420, 400], 1601, 501, 16, 0),                     # the same at odd widths
    ([200, 260, 512, 700], 328, 4100, 16, 17),               # large tiles, a last column tile that is cut
    ([200, 260, 512, 700], 4104, 328, 16, 17),               # large tiles for the gradient of the rows
    ([200, 260, 512, 700], 4101, 331, 16, 0),
    ([200, 260, 512, 700], 331, 4101, 1, 0),                 # the same at odd widths
    ([300, 290], 96, 16390, 16, 0),                          # large tiles, a short sum
    ([40] * 32, 136, 520, 64, 0),                            # small tiles
    ([9] * 40, 2056, 72, 16, 0),                             # few rows, 16 at a time
    ([20] * 40, 1000, 1100, 16, 0),                          # few rows, 32 at a time
    ([4000, 10], 72, 40, 16, 0),                             # many rows, few results
    ([2500] * 2, 136, 72, 256, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_products_by_every_rule(dev, case):
    counts, k, n, align, extra = CASES[case]
    print(f"case {case}: {CASES[case]}", flush=True)
    g = torch.Generator(device=dev).manual_seed(case)
    plan, offsets, used = _plan(counts, align, dev, extra)
    r, e = plan["r_cap"], len(counts)
    x, d, w = _rand(g, r, k), _rand(g, r, n), _rand(g, e, n, k)
    x[~used], d[~used] = float("nan"), float("nan")
    nan = lambda *s, dtype=torch.bfloat16: torch.full(s, float("nan"), dtype=dtype, device=dev)  # noqa: E731
    got = mtb.ep_bf16_grouped_gemm(x, w, plan, out=nan(r, n))
    _check_rows(got, lambda at: x[at].double(), lambda i: w[i].double().T.contiguous(), counts, offsets, used, k, 0.0, "gemm")
    got = mtb.ep_bf16_grouped_dgrad(d, w, plan, out=nan(r, k))
    _check_rows(got, lambda at: d[at].double(), lambda i: w[i].double(), counts, offsets, used, n, 0.0, "dgrad")
    for dtype, step in ((torch.bfloat16, 2.0 ** -8), (torch.float32, U)):
        got = mtb.ep_bf16_grouped_wgrad(d, x, plan, out=nan(e, n, k, dtype=dtype))
        for i, (c, o) in enumerate(zip(counts, offsets)):
            a, b = d[o:o + c].double().T.contiguous(), x[o:o + c].double()
            _near(got[i], a @ b, (c + 20) * U * (a.abs() @ b.abs()), ("wgrad", i), step)


MX_CASES = [(EDGES, 224, 264, 16, 40), (EDGES, 192, 3000, 1, 0), ([900] + [0] * 14 + [3], 1632, 640, 16, 300),
            ([380, 420, 400], 1632, 500, 16, 0), ([200, 260, 512, 700], 864, 4101, 16, 17), ([300, 290], 96, 16390, 16, 0),
            ([9] * 40, 2080, 72, 16, 0), ([120, 3, 400], 4128, 130, 16, 0), ([4000, 10], 96, 40, 16, 0), ([70] * 24, 800, 520, 64, 0)]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("case", range(len(MX_CASES)))
def test_mxfp4_products_by_every_rule(dev, case, eight):
    counts, k, n, align, extra = MX_CASES[case]
    print(f"mx case {case}: {MX_CASES[case]} {eight}", flush=True)
    g = torch.Generator(device=dev).manual_seed(case)
    plan, offsets, used = _plan(counts, align, dev, extra)
    r, e = plan["r_cap"], len(counts)
    x = _rand(g, r, k)
    x[:, : k // 2] *= 8.0
    wc, ws = (v.view(e, n, -1) for v in mtb.ep_mxfp4_pack(_rand(g, e * n, k)))
    if eight:
        data, s, _ = mtb.ep_mxfp8_pack(x)
        values = mtb.ep_mxfp8_unpack(data, s)
    else:
        data, s = mtb.ep_mxfp4_pack(x)
        values = mtb.ep_mxfp4_unpack(data, s)
    s[~used] = 255
    got = mtb.ep_mxfp4_grouped_gemm(data, s, wc, ws, plan, out=torch.full((r, n), float("nan"), dtype=torch.bfloat16, device=dev))
    _check_rows(got, lambda at: values[at].double(), lambda i: mtb.ep_mxfp4_unpack(wc[i], ws[i]).double().T.contiguous(), counts,
                offsets, used, k, 2.0 ** -10 if eight else 0.0, "product")


def test_plans_that_leave_spans_empty(dev):
    """Experts of a fixed room of which some hold nothing, and a plan whose room ends
    before the rows do: everything without an entry is zeros."""
    g = torch.Generator(device=dev).manual_seed(0)
    e, room, k, n = 6, 48, 72, 40
    counts = torch.tensor([0, 5, 48, 0, 47, 0], dtype=torch.int32, device=dev)
    offsets = (torch.arange(e + 1, device=dev) * room).int()
    r = e * room + 600
    plan = dict(counts=counts, offsets=offsets, dst_row=torch.zeros((100, 1), dtype=torch.int32, device=dev),
                src_row=torch.zeros(r, dtype=torch.int32, device=dev), r_cap=r, num_experts=e, alignment=16)
    used = torch.zeros(r, dtype=torch.bool, device=dev)
    for i, c in enumerate(counts.tolist()):
        used[i * room:i * room + c] = True
    x, d, w = _rand(g, r, k), _rand(g, r, n), _rand(g, e, n, k)
    c, o = counts.tolist(), offsets.tolist()[:-1]
    _check_rows(mtb.ep_bf16_grouped_gemm(x, w, plan), lambda at: x[at].double(), lambda i: w[i].double().T.contiguous(), c, o,
                used, k, 0.0, "gemm")
    _check_rows(mtb.ep_bf16_grouped_dgrad(d, w, plan), lambda at: d[at].double(), lambda i: w[i].double(), c, o, used, n, 0.0,
                "dgrad")
    dw = mtb.ep_bf16_grouped_wgrad(d, x, plan)
    assert not bool(dw[counts == 0].any()) and bool(dw[1].any())


def test_a_workspace_of_ones_own(dev):
    """The shares' workspace handed over: as large as asked for, smaller refused, and the
    same results as with one of the call's."""
    g = torch.Generator(device=dev).manual_seed(3)
    plan, offsets, used = _plan([3000, 2500], 16, dev)
    r, k, n = plan["r_cap"], 136, 72
    x, d = _rand(g, r, k), _rand(g, r, n)
    need = mtb.ep_bf16_grouped_wgrad_workspace_bytes(n, k, 2, plan["dst_row"].numel())
    assert need > 0
    want = mtb.ep_bf16_grouped_wgrad(d, x, plan, dtype=torch.float32)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev)
    assert torch.equal(mtb.ep_bf16_grouped_wgrad(d, x, plan, dtype=torch.float32, workspace=ws), want)
    with pytest.raises(ValueError):
        mtb.ep_bf16_grouped_wgrad(d, x, plan, workspace=ws[:-1])
    with pytest.raises(mtb.EpError):
        mtb.ep_bf16_grouped_wgrad(d, x, plan, workspace=torch.zeros(need + 1, dtype=torch.uint8, device=dev)[1:])


@pytest.mark.parametrize("room", [48, 300])
def test_plans_without_entries(dev, room):
    """No tokens at all, but grouped rows: zeros from every product."""
    e, k, n = 3, 96, 40
    plan = mtb.ep_route_plan(torch.zeros((0, 2), dtype=torch.int32, device=dev), e, 16, r_cap=room)
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device=dev)  # noqa: E731
    u8 = lambda *s: torch.full(s, 255, dtype=torch.uint8, device=dev)  # noqa: E731
    w = torch.ones((e, n, k), dtype=torch.bfloat16, device=dev)
    wc, ws = (v.view(e, n, -1) for v in mtb.ep_mxfp4_pack(w.view(-1, k)))
    for name, call in (("gemm", lambda: mtb.ep_bf16_grouped_gemm(nan(room, k), w, plan, out=nan(room, n))),
                       ("dgrad", lambda: mtb.ep_bf16_grouped_dgrad(nan(room, n), w, plan, out=nan(room, k))),
                       ("wgrad", lambda: mtb.ep_bf16_grouped_wgrad(nan(room, n), nan(room, k), plan, out=nan(e, n, k))),
                       ("mx4", lambda: mtb.ep_mxfp4_grouped_gemm(u8(room, k // 2), u8(room, k // 32), wc, ws, plan, out=nan(room, n))),
                       ("mx8", lambda: mtb.ep_mxfp4_grouped_gemm(u8(room, k), u8(room, k // 32), wc, ws, plan, out=nan(room, n)))):
        print(name, flush=True)
        got = call()
        assert not bool(got.view(torch.int16).any()), name
