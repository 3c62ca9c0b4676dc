"""The expert layer's steps on the GPU against the float64 oracle: BF16 dispatch
and combine with their gradients, the products with NVFP4 weights, SwiGLU with its
8-bit checkpoint.

Bars: a BF16 result is the rounding of a value within these of the float64 one,
with u = 2^-24 (FP32):
* a sum of n terms in FP32, in any order and with any fused steps, is within
  (n + 1) u of the sum of the terms' magnitudes;
* sigmoid(a) by exp and reciprocal instructions of 1 ulp each: the exponent
  a log2(e) is rounded once, so its relative error is below (|a| + 16) 2^-22;
  below -87, where exp(-a) leaves FP32's range, it is below 2^-120 and may be 0;
* copies and MXFP8 bytes are equal bit for bit.
"""

import numpy as np
import pytest
import torch

import moe_token_block_amd as mtb
from oracle import dswiglu as odsw
from oracle import expert, mxfp8, nvfp4
from oracle import formats as F
from oracle.routing import route_plan as o_route

from gpu_util import require_gpu, bf16_dev, host, i32_dev, assert_bytes_equal

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _bits(x):
    return F.f32_to_bf16(np.asarray(x, dtype=np.float32))


def _near(got_bits, want, slack, what):
    """BF16 results that are the rounding of something within ``slack`` of float64
    values: rounding keeps order, so they lie between the rounded ends."""
    got = expert.f64(host(got_bits) if torch.is_tensor(got_bits) else got_bits)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    with np.errstate(over="ignore"):
        lo, hi = expert.f64(odsw.f64_to_bf16(want - slack)), expert.f64(odsw.f64_to_bf16(want + slack))
    bad = ~((got >= lo) & (got <= hi))
    if bad.any():
        i = tuple(b[0] for b in np.nonzero(bad))
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; first at {i}: {got[i]} want {want[i]} "
                             f"slack {slack[i] if np.ndim(slack) else slack}")


def _ids(rng, t, e, k, drop):
    ids = np.argsort(rng.standard_normal((t, e)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random(ids.shape) < drop] = -1
    return ids


def _plan(ids, e, align, dev):
    return mtb.ep_route_plan(torch.from_numpy(np.ascontiguousarray(ids)).to(dev), e, align)


# tokens, experts, top_k, hidden, alignment, share of dropped slots
ROUTES = [(1, 8, 2, 4096, 16, 0.0), (1, 2, 1, 1, 16, 0.0), (3, 4, 4, 7, 16, 0.3), (5, 3, 2, 8, 16, 1.0),
          (17, 5, 3, 9, 32, 0.2), (33, 16, 8, 520, 16, 0.1), (40, 12, 9, 1001, 16, 0.2), (130, 20, 17, 72, 16, 0.1),
          (64, 4, 1, 7168, 128, 0.0), (257, 7, 3, 513, 16, 0.5), (29, 64, 5, 2056, 16, 0.0), (2, 8, 2, 16387, 16, 0.0),
          (300, 3, 2, 2, 16, 0.1), (21, 6, 2, 4099, 16, 0.1)]


# ------------------------------------------------------------------ dispatch, combine, gradients
@pytest.mark.parametrize("case", ROUTES)
def test_dispatch_combine_and_gradients(dev, case):
    t, e, k, h, align, drop = case
    rng = np.random.default_rng(t * h + k)
    ids = _ids(rng, t, e, k, drop)
    op = o_route(ids, e, align)
    dst, src = op["dst_row"], op["src_row"]
    plan = _plan(ids, e, align, dev)
    r = len(src)
    x, rows, dout = (_bits(rng.standard_normal(s)) for s in ((t, h), (r, h), (t, h)))
    rows[src < 0] = 0x7FC0                       # padding holds NaN: it may not be read
    w = rng.standard_normal((t, k)).astype(np.float32)
    w[dst < 0] = np.nan                          # the weight of an unused slot is not used
    print(f"rows {case}", flush=True)
    assert_bytes_equal(host(mtb.ep_bf16_dispatch(bf16_dev(x, dev), plan)), expert.dispatch(x, src), "dispatch")
    want, mag = expert.combine(expert.f64(rows), dst, w)
    wd, rd = torch.from_numpy(w).to(dev), bf16_dev(rows, dev)
    got = mtb.ep_bf16_combine(rd, plan, wd)
    _near(got, want, (k + 1) * U * mag, "combine")
    want, mag = expert.combine(expert.f64(rows), dst)
    _near(mtb.ep_bf16_combine(rd, plan), want, (k + 1) * U * mag, "combine without weights")
    want, dw, mag = expert.combine_bwd(expert.f64(dout), expert.f64(rows), dst, w)
    drows, dweights = mtb.ep_bf16_combine_bwd(bf16_dev(dout, dev), rd, plan, wd)
    _near(drows, want, U * np.abs(want), "drows")
    assert np.all(np.abs(host(dweights) - dw) <= (h + 1) * U * mag), "dweights"
    assert not host(dweights)[dst < 0].any()
    assert not host(drows)[src < 0].any()


def test_rows_of_no_tokens_and_of_no_rows(dev):
    for t in (0, 4):
        ids = np.full((t, 2), -1, dtype=np.int32)
        plan = _plan(ids, 3, 16, dev)
        h = 40
        out = mtb.ep_bf16_dispatch(torch.zeros((t, h), dtype=torch.bfloat16, device=dev), plan)
        assert not host(out).any() and out.shape == (plan["r_cap"], h)
        rows = torch.full((plan["r_cap"], h), float("nan"), dtype=torch.bfloat16, device=dev)
        w = torch.full((t, 2), float("inf"), device=dev)
        assert not host(mtb.ep_bf16_combine(rows, plan, w)).any()
        drows, dw = mtb.ep_bf16_combine_bwd(torch.ones((t, h), dtype=torch.bfloat16, device=dev), rows, plan, w)
        assert not host(drows).any() and not host(dw).any()


def test_special_values_follow_the_formula(dev):
    # inf and NaN in rows that are used reach their token only, a zero weight included
    ids = np.array([[0, 1], [1, 0], [0, 1]], dtype=np.int32)
    plan = _plan(ids, 2, 16, dev)
    dst = host(plan["dst_row"])
    h = 24
    rows = np.ones((plan["r_cap"], h), dtype=np.float32)
    rows[dst[0, 0], 3] = np.inf
    rows[dst[1, 1], 5] = np.nan
    w = np.array([[0.0, 2.0], [1.0, 0.0], [0.25, 0.5]], dtype=np.float32)
    got = expert.f64(host(mtb.ep_bf16_combine(bf16_dev(_bits(rows), dev), plan, torch.from_numpy(w).to(dev))))
    with np.errstate(invalid="ignore"):
        want = (w[:, :, None] * rows[dst]).sum(1)
    np.testing.assert_array_equal(got, want)


def test_maps_that_point_outside_are_skipped(dev):
    # a plan's own maps never do: the kernels' bounds hold for any others
    t, k, h, r = 3, 2, 32, 48
    rng = np.random.default_rng(0)
    dst = np.array([[0, 48], [2 ** 31 - 1, 1], [-5, -(2 ** 31)]], dtype=np.int64).astype(np.int32)
    src = np.full(r, 3, dtype=np.int32)          # no token 3
    src[0], src[1] = 0, 1
    plan = dict(counts=i32_dev([2], dev), offsets=i32_dev([0, 48], dev), src_row=i32_dev(src, dev),
                dst_row=i32_dev(dst, dev), r_cap=r, num_experts=1)
    x, rows, dout = (_bits(rng.standard_normal(s)) for s in ((t, h), (r, h), (t, h)))
    w = rng.standard_normal((t, k)).astype(np.float32)
    wd, rd = torch.from_numpy(w).to(dev), bf16_dev(rows, dev)
    assert_bytes_equal(host(mtb.ep_bf16_dispatch(bf16_dev(x, dev), plan)), expert.dispatch(x, src), "dispatch")
    want, mag = expert.combine(expert.f64(rows), dst, w)
    _near(mtb.ep_bf16_combine(rd, plan, wd), want, (k + 1) * U * mag, "combine")
    want, dw, mag = expert.combine_bwd(expert.f64(dout), expert.f64(rows), dst, w)
    drows, dweights = mtb.ep_bf16_combine_bwd(bf16_dev(dout, dev), rd, plan, wd)
    _near(drows, want, U * np.abs(want), "drows")
    assert np.all(np.abs(host(dweights) - dw) <= (h + 1) * U * mag)


def test_rows_past_32_bit_offsets(dev):
    # grouped rows whose element offsets pass 2^31 and byte offsets 2^32
    h, r, t, k = 7168, 330000, 3, 2
    dst = np.array([[r - 1, 0], [299593, 5], [r - 2, 299594]], dtype=np.int32)
    src = np.full(r, -1, dtype=np.int32)
    src[dst.reshape(-1)] = np.repeat(np.arange(t), k)
    plan = dict(counts=i32_dev([r], dev), offsets=i32_dev([0, r], dev), src_row=i32_dev(src, dev),
                dst_row=i32_dev(dst, dev), r_cap=r, num_experts=1)
    rng = np.random.default_rng(1)
    x, dout, used = (_bits(rng.standard_normal((n, h))) for n in (t, t, t * k))
    w = rng.standard_normal((t, k)).astype(np.float32)
    at = torch.from_numpy(dst.reshape(-1)).long().to(dev)
    out = mtb.ep_bf16_dispatch(bf16_dev(x, dev), plan)
    assert_bytes_equal(host(out[at]), np.repeat(x, k, axis=0), "dispatch")
    assert int(torch.count_nonzero(out.view(torch.int16)).item()) == np.count_nonzero(x) * k
    out[at] = bf16_dev(used, dev)
    small = np.arange(t * k, dtype=np.int32).reshape(t, k)
    wd = torch.from_numpy(w).to(dev)
    want, mag = expert.combine(expert.f64(used), small, w)
    _near(mtb.ep_bf16_combine(out, plan, wd), want, (k + 1) * U * mag, "combine")
    want, dw, mag = expert.combine_bwd(expert.f64(dout), expert.f64(used), small, w)
    drows, dweights = mtb.ep_bf16_combine_bwd(bf16_dev(dout, dev), out, plan, wd)
    _near(drows[at], want, U * np.abs(want), "drows")
    assert np.all(np.abs(host(dweights) - dw) <= (h + 1) * U * mag)
    drows[at] = 0
    assert not bool(drows.view(torch.int16).any().item())


# ------------------------------------------------------------------ NVFP4 matrix-vector products
def _weights(rng, e, n, k):
    w = rng.standard_normal((e * n, k)) / np.sqrt(k) * 2.0 ** rng.integers(-6, 7, size=(e * n, 1))
    w[rng.integers(0, e * n)] = 0.0              # a zero row: t = 1, scales 0
    w[rng.integers(0, e * n), :16] = 0.0         # a zero block
    return nvfp4.pack_rows(_bits(w)).reshape(e, n, -1)


def _check_matvec(got, x, weight, ids, swiglu, what):
    K = x.shape[-1]
    y, mag = expert.matvec(x, weight, ids)
    err = 2 * (K + 1) * U * mag                  # the matrix instruction's own order may round twice a term
    if swiglu:
        g, u = np.split(y, 2, axis=-1)
        eg, eu = np.split(err, 2, axis=-1)
        s = g * expert.sigmoid(g)
        err = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + np.abs(s * u) * (np.abs(g) + 16) * 2.0 ** -22
        err += np.abs(u) * 2.0 ** -110
        y = s * u
    _near(got, y, err, what)


# tokens, experts, top_k, width, hidden, dropped, per entry, swiglu
MATVEC = [(1, 8, 2, 64, 4096, 0.0, False, True), (1, 1, 1, 1, 64, 0.0, False, False), (1, 4, 3, 17, 128, 0.4, True, False),
          (2, 3, 2, 33, 192, 0.0, False, False), (5, 2, 2, 50, 1088, 0.2, True, True), (7, 32, 8, 16, 320, 0.1, False, False),
          (16, 2, 1, 40, 256, 0.0, False, True), (17, 3, 2, 35, 704, 0.0, True, False), (33, 2, 2, 24, 576, 0.1, False, True),
          (64, 5, 3, 70, 448, 0.0, False, False), (100, 1, 1, 130, 64, 0.0, False, False), (128, 4, 4, 18, 2048, 0.3, True, True),
          (3, 7, 4, 260, 7168, 0.0, False, False), (50, 2, 1, 37, 1600, 0.0, False, False), (70, 1, 1, 44, 512, 0.0, True, True),
          (97, 2, 2, 300, 576, 0.1, False, False), (7, 1, 1, 129, 64, 0.0, False, False), (4, 8, 2, 4098, 640, 0.0, False, True),
          (9, 2, 2, 18, 4160, 0.0, True, False), (200, 3, 1, 514, 1088, 0.05, False, True), (9, 5, 5, 8, 832, 1.0, False, False), (1000, 6, 4, 6, 128, 0.1, False, True)]


@pytest.mark.parametrize("case", MATVEC)
def test_expert_matvec(dev, case):
    t, e, k, n, K, drop, per, swiglu = case
    rng = np.random.default_rng(t * n + K)
    ids = _ids(rng, t, e, k, drop)
    weight = _weights(rng, e, n, K)
    xb = _bits(rng.standard_normal((t, k, K) if per else (t, K)) * 10.0 ** rng.uniform(-2, 2))
    xb.reshape(-1)[:: 37] = 0
    print(f"matvec {case}", flush=True)
    wd = torch.from_numpy(weight).to(dev)
    got = mtb.ep_nvfp4_expert_matvec(bf16_dev(xb, dev), wd, torch.from_numpy(ids).to(dev), swiglu=swiglu)
    _check_matvec(got, expert.f64(xb), weight, ids, swiglu, f"matvec {case}")
    assert not host(got)[ids < 0].any()
    again = mtb.ep_nvfp4_expert_matvec(bf16_dev(xb, dev), wd, torch.from_numpy(ids.astype(np.int64)).to(dev),
                                       swiglu=swiglu)
    assert_bytes_equal(host(again), host(got), "the same call with 64-bit ids")


# Entries of each expert (and of none), width, hidden, swiglu.  First widths at which four waves side by side
# fill the GPU: passes of one to four column tiles, more than one pass, an empty expert; then few rows of
# weights, whose entries several blocks share out, some in more than one turn.
SHARES = [([1, 17, 33, 49, 64, 65, 150, 0, 16, 2, 3, 48, 5, 6, 32, 7], 9, 2050, 576, False),
          ([1, 17, 33, 49, 64, 65, 150, 0, 16, 2, 3, 48, 5, 6, 32, 7], 0, 2050, 1088, True),
          ([130, 70, 31, 1, 16, 17, 0, 8], 3, 4030, 64, False),
          ([200, 0, 40], 5, 40, 7168, False), ([200, 1, 39], 0, 42, 1600, True),
          ([230, 0, 10], 2, 1300, 1088, False), ([16, 300, 33], 0, 700, 2112, True), ([40, 4000], 30, 3, 128, False)]


@pytest.mark.parametrize("case", SHARES)
def test_matvec_with_uneven_experts(dev, case):
    counts, none, n, K, swiglu = case
    rng = np.random.default_rng(n + K)
    ids = np.repeat(np.arange(-1, len(counts)), [none] + counts).astype(np.int32)
    rng.shuffle(ids)
    ids = ids[:, None]
    weight = _weights(rng, len(counts), n, K)
    xb = _bits(rng.standard_normal((ids.size, K)))
    print(f"matvec {case}", flush=True)
    xd, wd, idd = bf16_dev(xb, dev), torch.from_numpy(weight).to(dev), torch.from_numpy(ids).to(dev)
    got = mtb.ep_nvfp4_expert_matvec(xd, wd, idd, swiglu=swiglu)
    _check_matvec(got, expert.f64(xb), weight, ids, swiglu, f"matvec {case}")
    assert not host(got)[ids < 0].any()
    wo = torch.empty(wd.numel() + 8, dtype=torch.uint8, device=dev)[3 : 3 + wd.numel()].view(wd.shape)
    xo = torch.empty(xd.numel() + 8, dtype=torch.bfloat16, device=dev)[1 : 1 + xd.numel()].view(xd.shape)
    wo.copy_(wd)
    xo.copy_(xd)
    assert_bytes_equal(host(mtb.ep_nvfp4_expert_matvec(xo, wo, idd.long(), swiglu=swiglu)), host(got), "odd addresses")


@pytest.mark.parametrize("t,n,K,swiglu", [(1, 1, 64, False), (1, 4096, 128, True), (3, 1001, 1088, False),
                                          (20, 77, 960, False), (130, 34, 192, True), (2, 16, 16384, False)])
def test_dense_matvec(dev, t, n, K, swiglu):
    rng = np.random.default_rng(n + K)
    weight = _weights(rng, 1, n, K)[0]
    xb = _bits(rng.standard_normal((t, K)))
    print(f"dense {t} {n} {K}", flush=True)
    got = mtb.ep_nvfp4_expert_matvec(bf16_dev(xb, dev), torch.from_numpy(weight).to(dev), swiglu=swiglu)
    _check_matvec(got, expert.f64(xb), weight, None, swiglu, "dense")


@pytest.mark.parametrize("t,e,k,swiglu", [(3, 4, 2, False), (40, 2, 2, True)])  # few and many entries an expert
def test_matvec_at_any_address(dev, t, e, k, swiglu):
    rng = np.random.default_rng(t)
    weight, ids = _weights(rng, e, 50, 1088), _ids(rng, t, e, k, 0.1)
    xb = _bits(rng.standard_normal((t, 1088)))
    wd, xd, idd = torch.from_numpy(weight).to(dev), bf16_dev(xb, dev), torch.from_numpy(ids).to(dev)
    base = mtb.ep_nvfp4_expert_matvec(xd, wd, idd, swiglu=swiglu)
    _check_matvec(base, expert.f64(xb), weight, ids, swiglu, "aligned")
    for off in (1, 2, 3, 7):
        wo = torch.empty(wd.numel() + 8, dtype=torch.uint8, device=dev)[off : off + wd.numel()].view(wd.shape)
        xo = torch.empty(xd.numel() + 8, dtype=torch.bfloat16, device=dev)[off : off + xd.numel()].view(xd.shape)
        wo.copy_(wd)
        xo.copy_(xd)
        assert_bytes_equal(host(mtb.ep_nvfp4_expert_matvec(xo, wo, idd, swiglu=swiglu)), host(base), f"offset {off}")


def test_matvec_drops_and_flags_bad_ids(dev):
    rng = np.random.default_rng(11)
    weight = _weights(rng, 3, 20, 128)
    xb = _bits(rng.standard_normal((4, 128)))
    ids = np.array([[0, 3], [-1, 1], [2, -2], [2 ** 31 - 1, 1]], dtype=np.int64)
    ids[3, 0] = 2 ** 33                           # 0 in its low 32 bits
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    got = mtb.ep_nvfp4_expert_matvec(bf16_dev(xb, dev), torch.from_numpy(weight).to(dev),
                                     torch.from_numpy(ids).to(dev), d_error=err)
    _check_matvec(got, expert.f64(xb), weight, ids, False, "bad ids")
    assert int(err.item()) == mtb.EP_DEVERR_EXPERT_ID
    err.zero_()
    good = np.where((ids >= 0) & (ids < 3), ids, -1)
    mtb.ep_nvfp4_expert_matvec(bf16_dev(xb, dev), torch.from_numpy(weight).to(dev), torch.from_numpy(good).to(dev),
                               d_error=err)
    assert int(err.item()) == 0


def test_matvec_special_values_stay_in_their_row(dev):
    # NaN and inf of one token's row, and of rows that only unused slots name, reach no other token
    rng = np.random.default_rng(12)
    weight = _weights(rng, 2, 24, 256)
    x = rng.standard_normal((6, 256)).astype(np.float32)
    x[1, 7], x[4, 0] = np.nan, np.inf
    ids = np.array([[0, 1], [1, 0], [0, -1], [1, 0], [-1, -1], [0, 1]], dtype=np.int32)
    got = expert.f64(host(mtb.ep_nvfp4_expert_matvec(bf16_dev(_bits(x), dev), torch.from_numpy(weight).to(dev),
                                                     torch.from_numpy(ids).to(dev))))
    clean = x.copy()
    clean[1], clean[4] = 0, 0
    y, mag = expert.matvec(expert.f64(_bits(clean)), weight, ids)
    keep = [0, 2, 3, 4, 5]
    assert np.isnan(got[1]).all()
    _near(_bits(got[keep]), y[keep], (2 * 257 * U * mag)[keep], "other rows")


@pytest.mark.parametrize("scale,x_scale", [(2.0 ** -115, 2.0 ** 115), (2.0 ** 100, 2.0 ** -100), (2.0 ** -128, 2.0 ** 120)])
def test_matvec_far_from_one(dev, scale, x_scale):
    # weight rows and activations at the ends of BF16's range (row scales below FP32's normal numbers in the last)
    # whose products are ordinary numbers
    rng = np.random.default_rng(13)
    w = nvfp4.pack_rows(_bits(rng.standard_normal((24, 192)) * scale)).reshape(1, 24, -1)
    xb = _bits(rng.standard_normal((3, 192)) * x_scale)
    ids = np.zeros((3, 1), dtype=np.int32)
    got = mtb.ep_nvfp4_expert_matvec(bf16_dev(xb, dev), torch.from_numpy(w).to(dev), torch.from_numpy(ids).to(dev))
    _check_matvec(got, expert.f64(xb), w, ids, False, f"scale {scale}")


# ------------------------------------------------------------------ SwiGLU and its 8-bit checkpoint
def _act_slack(p):
    a, b = np.split(p, 2, axis=-1)
    return np.abs(expert.swiglu(p)) * (np.abs(a) + 16) * 2.0 ** -22 + np.abs(b) * 2.0 ** -110


def _grad_slack(p, dy):
    a, b = np.split(p, 2, axis=-1)
    s = expert.sigmoid(a)
    rel = (np.abs(a) + 16) * 2.0 ** -22
    da = np.abs(dy * b) * (s * (1 + np.abs(a)) * rel + (1 + np.abs(a)) * 2.0 ** -120)
    db = np.abs(dy) * (np.abs(a) * s * rel + np.abs(a) * 2.0 ** -120)
    return np.concatenate([da, db], axis=-1)


@pytest.mark.parametrize("t,f", [(1, 32), (1, 2048), (3, 96), (5, 1024), (7, 1056), (33, 64), (64, 320), (257, 32), (2, 14336)])
def test_swiglu_checkpoint_and_gradient(dev, t, f):
    rng = np.random.default_rng(t * f)
    p = rng.standard_normal((t, 2 * f)) * 10.0 ** rng.uniform(-2, 1.5, size=(t, 1))
    p[0, :32] = 0.0                               # a zero block
    p[-1, f : f + 32] *= 2.0 ** -100              # a block far below the others
    p[-1, f - 32 : f : 5] = -0.0
    pb, dyb = _bits(p), _bits(rng.standard_normal((t, f)) * 1e-2)
    print(f"swiglu {t} x {f}", flush=True)
    act, data, scales = mtb.swiglu_mxfp8_checkpoint(bf16_dev(pb, dev))
    _near(act, expert.swiglu(expert.f64(pb)), _act_slack(expert.f64(pb)), "act")
    want_data, want_scales = mxfp8.pack_rows(pb)
    assert_bytes_equal(host(data), want_data, "checkpoint data")
    assert_bytes_equal(host(scales), want_scales, "checkpoint scales")
    v = mxfp8.decode(want_data, want_scales)
    assert_bytes_equal(host(mtb.ep_mxfp8_unpack(data, scales)), odsw.f64_to_bf16(v), "unpacked checkpoint")
    dx, act2 = mtb.dswiglu_mxfp8_checkpoint(data, scales, bf16_dev(dyb, dev))
    dy = expert.f64(dyb)
    _near(dx, expert.swiglu_grad(v, dy), _grad_slack(v, dy), "dx")
    _near(act2, expert.swiglu(v), _act_slack(v), "act from the checkpoint")
    dx2, none = mtb.dswiglu_mxfp8_checkpoint(data, scales, bf16_dev(dyb, dev), need_act=False)
    assert none is None
    assert_bytes_equal(host(dx2), host(dx), "dx without act")


def test_swiglu_gradient_against_differences(dev):
    # the kernel's dx times a step is the change of the loss that the float64 forward sees:
    # |step| is a power of two small enough for second-order terms (|silu''| < 1) to stay below BF16's rounding
    rng = np.random.default_rng(8)
    t, f = 6, 64
    data, scales = mxfp8.pack_rows(_bits(rng.standard_normal((t, 2 * f))))
    v, dyb = mxfp8.decode(data, scales), _bits(rng.standard_normal((t, f)))
    dx, _ = mtb.dswiglu_mxfp8_checkpoint(torch.from_numpy(data).to(dev), torch.from_numpy(scales).to(dev),
                                         bf16_dev(dyb, dev))
    dy, h = expert.f64(dyb), 2.0 ** -17
    a, b = np.split(v, 2, axis=1)
    one = lambda q: expert.swiglu(q) * dy
    da = (one(np.concatenate([a + h, b], 1)) - one(np.concatenate([a - h, b], 1))) / (2 * h)
    db = (one(np.concatenate([a, b + h], 1)) - one(np.concatenate([a, b - h], 1))) / (2 * h)
    want = np.concatenate([da, db], 1)
    slack = _grad_slack(v, dy) + 2.0 ** -34 * np.concatenate([np.abs(dy * b), np.abs(dy)], 1) + 2.0 ** -34
    _near(dx, want, slack, "dx against differences")


def test_swiglu_extreme_gates(dev):
    f = 32
    a = np.array([0.0, -0.0, 1e-38, 20.0, -20.0, 60.0, -60.0, 86.0, -86.0, 120.0, -120.0, 3e4, -3e4, 1e30, -1e30, 88.5], dtype=np.float32)
    p = np.zeros((1, 2 * f), dtype=np.float32)
    p[0, :16], p[0, 16:32] = a, -a
    p[0, f:] = np.linspace(-2, 2, f)
    pb = _bits(p)
    act, _, _ = mtb.swiglu_mxfp8_checkpoint(bf16_dev(pb, dev))
    v = expert.f64(pb)
    _near(act, expert.swiglu(v), _act_slack(v), "extreme gates")


@pytest.mark.parametrize("h", [32, 96, 4096])
def test_unpack_every_byte(dev, h):
    rng = np.random.default_rng(h)
    rows = 512
    data = rng.integers(0, 256, size=(rows, h)).astype(np.uint8)
    scales = rng.integers(0, 256, size=(rows, h // 32)).astype(np.uint8)
    scales[:256, 0] = np.arange(256)
    data[0::2, :32] = np.arange(rows // 2, dtype=np.uint8)[:, None]
    got = host(mtb.ep_mxfp8_unpack(torch.from_numpy(data).to(dev), torch.from_numpy(scales).to(dev)))
    nan = ((data & 0x7F) == 0x7F) | np.repeat(scales == 255, 32, axis=1)
    v = F.e4m3_decode(np.where(nan, 0, data).astype(np.uint8)) * np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)
    v = np.where(nan, 0.0, v)
    huge = np.abs(v) >= 2.0 ** 128 * (1 - 2.0 ** -9)           # past BF16's largest, or rounded there
    want = odsw.f64_to_bf16(np.where(huge, 0.0, v))
    want = np.where(huge, np.where(v < 0, 0xFF80, 0x7F80), want).astype(np.uint16)
    sign = (data & 0x80).astype(np.uint16) << 8
    assert_bytes_equal(got[~nan] | 0, (want | sign)[~nan], "unpack")
    assert np.all((got[nan] & 0x7FFF) > 0x7F80), "NaN"


# ------------------------------------------------------------------ streams, views, graphs, refusals
def test_views_streams_and_given_outputs(dev):
    rng = np.random.default_rng(20)
    t, e, k, h = 19, 4, 2, 136
    ids = _ids(rng, t, e, k, 0.1)
    plan = _plan(ids, e, 16, dev)

    def odd(a, dtype):
        """The same values at an odd element offset of a larger buffer."""
        buf = torch.empty(a.numel() + 3, dtype=dtype, device=dev)
        v = buf[3 : 3 + a.numel()].view(a.shape)
        v.copy_(a)
        return v

    x, rows, dout = (torch.randn(n, h, device=dev).bfloat16() for n in (t, plan["r_cap"], t))
    w = torch.rand(t, k, device=dev)
    F_ = 96
    pre, dy = torch.randn(t, 2 * F_, device=dev).bfloat16(), torch.randn(t, F_, device=dev).bfloat16()
    weight = torch.from_numpy(_weights(rng, e, 30, 128)).to(dev)
    xs = torch.randn(t, 128, device=dev).bfloat16()
    idd = torch.from_numpy(ids).to(dev)

    def everything(f, outs):
        o = outs.pop if outs else lambda: None
        res = [mtb.ep_bf16_dispatch(f(x), plan, out=o()), mtb.ep_bf16_combine(f(rows), plan, w, out=o())]
        res += mtb.ep_bf16_combine_bwd(f(dout), f(rows), plan, w, drows=o(), dweights=o())
        res.append(mtb.ep_nvfp4_expert_matvec(f(xs), f(weight), idd, swiglu=True, out=o()))
        res += mtb.swiglu_mxfp8_checkpoint(f(pre), act=o(), data=o(), scales=o())
        data, scales = res[-2], res[-1]
        res.append(mtb.ep_mxfp8_unpack(data, scales, out=o()))
        res += mtb.dswiglu_mxfp8_checkpoint(data, scales, f(dy), dx=o(), act=o())
        return res

    base = everything(lambda a: a, [])
    torch.cuda.synchronize(dev)
    got = everything(lambda a: odd(a, a.dtype), [odd(torch.zeros_like(b), b.dtype) for b in reversed(base)])
    for i, (a, b) in enumerate(zip(got, base)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"output {i} at an odd address"
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        got = everything(lambda a: a, [])
    side.synchronize()
    for i, (a, b) in enumerate(zip(got, base)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"output {i} on another stream"


def test_graph_capture_replays(dev):
    rng = np.random.default_rng(21)
    t, e, k, h = 12, 4, 2, 256
    plan = _plan(_ids(rng, t, e, k, 0.1), e, 16, dev)
    ids = torch.from_numpy(_ids(rng, t, e, k, 0.1)).to(dev)
    w = torch.rand(t, k, device=dev)
    w1 = torch.from_numpy(_weights(rng, e, 128, h)).to(dev)
    w2 = torch.from_numpy(_weights(rng, e, h, 64)).to(dev)
    x = torch.randn(t, h, device=dev).bfloat16()

    def step():
        act = mtb.ep_nvfp4_expert_matvec(x, w1, ids, swiglu=True)
        y = mtb.ep_nvfp4_expert_matvec(act, w2, ids)
        rows = mtb.ep_bf16_dispatch(x, plan)
        out = mtb.ep_bf16_combine(rows, plan, w)
        drows, dw = mtb.ep_bf16_combine_bwd(out, rows, plan, w)
        a, data, scales = mtb.swiglu_mxfp8_checkpoint(drows)
        dx, _ = mtb.dswiglu_mxfp8_checkpoint(data, scales, a)
        return y, out, drows, dw, dx

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream(dev).wait_stream(side)
    torch.cuda.synchronize(dev)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(3):
        x.copy_(torch.randn(t, h, device=dev).bfloat16())
        g.replay()
        torch.cuda.synchronize(dev)
        for a, b in zip(out, step()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"replay {i}"


def test_results_do_not_depend_on_timing(dev):
    rng = np.random.default_rng(22)
    t, e, k, h = 700, 8, 3, 1024
    plan = _plan(_ids(rng, t, e, k, 0.05), e, 16, dev)
    rows = torch.randn(plan["r_cap"], h, device=dev).bfloat16()
    dout, w = torch.randn(t, h, device=dev).bfloat16(), torch.rand(t, k, device=dev)
    ids = torch.from_numpy(_ids(rng, 40, e, k, 0.0)).to(dev)
    weight = torch.from_numpy(_weights(rng, e, 48, 512)).to(dev)
    xs = torch.randn(40, 512, device=dev).bfloat16()
    first = None
    for _ in range(4):
        got = [*mtb.ep_bf16_combine_bwd(dout, rows, plan, w), mtb.ep_bf16_combine(rows, plan, w),
               mtb.ep_nvfp4_expert_matvec(xs, weight, ids, swiglu=True)]
        first = first or got
        for a, b in zip(got, first):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_binding_refusals(dev):
    plan = _plan(np.array([[0, 1], [1, 0]], dtype=np.int32), 2, 16, dev)
    r = plan["r_cap"]
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)
    f32 = lambda *s: torch.zeros(s, device=dev)
    ids = torch.zeros((2, 2), dtype=torch.int32, device=dev)
    rb = mtb.ep_nvfp4_packed_row_bytes(64)
    bad = [
        lambda: mtb.ep_bf16_dispatch(f32(2, 8), plan), lambda: mtb.ep_bf16_dispatch(bf(3, 8), plan),
        lambda: mtb.ep_bf16_dispatch(bf(2, 16)[:, ::2], plan), lambda: mtb.ep_bf16_dispatch(bf(2, 8), plan, out=bf(r, 9)),
        lambda: mtb.ep_bf16_dispatch(bf(2, 8).cpu(), plan),
        lambda: mtb.ep_bf16_combine(bf(r + 1, 8), plan), lambda: mtb.ep_bf16_combine(bf(r, 8), plan, f32(2, 3)),
        lambda: mtb.ep_bf16_combine(bf(r, 8), plan, bf(2, 2)), lambda: mtb.ep_bf16_combine(bf(r, 8), plan, out=bf(2, 7)),
        lambda: mtb.ep_bf16_combine_bwd(bf(2, 8), bf(r, 9), plan, f32(2, 2)),
        lambda: mtb.ep_bf16_combine_bwd(bf(3, 8), bf(r, 8), plan, f32(2, 2)),
        lambda: mtb.ep_bf16_combine_bwd(bf(2, 8), bf(r, 8), plan, f32(2, 2), dweights=f32(4)),
        lambda: mtb.ep_nvfp4_expert_matvec(bf(2, 64), u8(2, 4, rb + 1), ids),
        lambda: mtb.ep_nvfp4_expert_matvec(bf(2, 64), u8(2, 3, rb), ids, swiglu=True),
        lambda: mtb.ep_nvfp4_expert_matvec(bf(3, 64), u8(2, 4, rb), ids),
        lambda: mtb.ep_nvfp4_expert_matvec(bf(2, 3, 64), u8(2, 4, rb), ids),
        lambda: mtb.ep_nvfp4_expert_matvec(bf(2, 64), u8(2, 4, rb)),
        lambda: mtb.ep_nvfp4_expert_matvec(bf(2, 64), u8(2, 4, rb), ids.float()),
        lambda: mtb.ep_nvfp4_expert_matvec(bf(2, 64), u8(2, 4, rb), ids, out=bf(2, 2, 5)),
        lambda: mtb.ep_nvfp4_expert_matvec(bf(2, 96), u8(2, 4, 58), ids),
        lambda: mtb.swiglu_mxfp8_checkpoint(bf(2, 96)), lambda: mtb.swiglu_mxfp8_checkpoint(bf(2, 128), data=u8(2, 64)),
        lambda: mtb.swiglu_mxfp8_checkpoint(f32(2, 128)),
        lambda: mtb.dswiglu_mxfp8_checkpoint(u8(2, 128), u8(2, 4), bf(2, 128)),
        lambda: mtb.dswiglu_mxfp8_checkpoint(u8(2, 128), u8(2, 3), bf(2, 64)),
        lambda: mtb.dswiglu_mxfp8_checkpoint(u8(2, 96), u8(2, 3), bf(2, 48)),
        lambda: mtb.ep_mxfp8_unpack(u8(2, 40), u8(2, 1)), lambda: mtb.ep_mxfp8_unpack(u8(2, 64), u8(2, 2), out=bf(2, 32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, mtb.EpError)):
            call()
            raise AssertionError(f"call {i} was not refused")
    with pytest.raises(mtb.EpError):
        big = torch.zeros((2049, 2), dtype=torch.int32, device=dev)
        mtb.ep_nvfp4_expert_matvec(bf(2049, 64), u8(2, 4, rb), big)
