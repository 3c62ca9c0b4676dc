"""The expert layer's kernels for many entries, at sizes at which each rule picks
them: the combine and its gradient with streamed reads, the NVFP4 product of four
waves side by side.

Bounds are those of ``test_gpu_expert``; where a whole large result is compared on
the device, a BF16 result is within 2^-8 (half a unit in its last place) of what it
rounds."""

import numpy as np
import pytest
import torch

import moe_token_block_amd as mtb
from oracle import expert

from gpu_util import require_gpu, bf16_dev, host, assert_bytes_equal
from test_gpu_expert import U, _bits, _check_matvec, _ids, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


# ------------------------------------------------------------------ streamed reads
def _off_by_more(got, want, slack):
    return int(((got.double() - want).abs() > slack + 2.0 ** -8 * (want.abs() + slack)).sum())


# tokens, experts, top_k, hidden: entries * hidden above 2^27 values, two slots and more, whole and ragged pieces
@pytest.mark.parametrize("t,e,k,h", [(16900, 7, 2, 4101), (33000, 5, 1, 4096), (5900, 9, 5, 4611), (1400, 16, 9, 10800)])
@pytest.mark.parametrize("drop", [0.0, 0.2])
def test_combine_and_gradient_of_rows_past_the_caches(dev, t, e, k, h, drop):
    assert t * k * h * 2 > 256 << 20
    g = torch.Generator(device=dev).manual_seed(t + k)
    rng = np.random.default_rng(t)
    ids = torch.from_numpy(_ids(rng, t, e, k, drop)).to(dev)
    plan = mtb.ep_route_plan(ids, e, 16)
    dst, src = plan["dst_row"].long(), plan["src_row"]
    used = dst >= 0
    assert torch.equal(used, ids >= 0)
    rows = torch.randn(plan["r_cap"], h, generator=g, device=dev, dtype=torch.bfloat16)
    rows[src < 0] = float("nan")                 # padding holds NaN: it may not be read
    w = torch.rand(t, k, generator=g, device=dev).masked_fill(~used, float("nan"))
    dout = torch.randn(t, h, generator=g, device=dev, dtype=torch.bfloat16)
    print(f"streamed {t} x {h} top-{k}", flush=True)
    out, plain = mtb.ep_bf16_combine(rows, plan, w), mtb.ep_bf16_combine(rows, plan)
    drows, dweights = mtb.ep_bf16_combine_bwd(dout, rows, plan, w)
    assert not bool(drows[src < 0].view(torch.int16).any()) and not bool(dweights[~used].any())
    sums = [torch.zeros(t, h, dtype=torch.float64, device=dev) for _ in range(4)]
    d64 = dout.double()
    for j in range(k):
        on, at = used[:, j], dst[used[:, j], j]
        r, wj = rows[at].double(), w[on, j].double()[:, None]
        for s, term in zip(sums, (wj * r, (wj * r).abs(), r, r.abs())):
            s[on] += term
        assert _off_by_more(drows[at], wj * d64[on], U * (wj * d64[on]).abs()) == 0, f"drows of slot {j}"
        p = d64[on] * r
        off = (dweights[on, j].double() - p.sum(1)).abs() > (h + 1) * U * p.abs().sum(1)
        assert not bool(off.any()), f"dweights of slot {j}"
    assert _off_by_more(out, sums[0], (k + 1) * U * sums[1]) == 0, "combine"
    assert _off_by_more(plain, sums[2], (k + 1) * U * sums[3]) == 0, "combine without weights"


# ------------------------------------------------------------------ NVFP4 products, many entries an expert
def _many(t, e, k, n, swiglu):
    """Enough entries an expert and enough columns for blocks of four waves side by side."""
    cols = n // 2 if swiglu else n
    return t * k >= 16 * e and -(-cols // (64 if swiglu else 128)) * e >= 256


# tokens, experts, top_k, width, hidden, dropped, per entry, swiglu
MANY = [(130, 8, 2, 4000, 128, 0.0, False, False), (100, 16, 8, 1990, 192, 0.1, True, False),
        (90, 16, 3, 2020, 576, 0.05, False, True), (70, 16, 4, 2022, 64, 0.0, True, True),
        (150, 32, 8, 1000, 1088, 0.3, False, False), (33, 2, 1, 16370, 64, 0.0, False, False)]


@pytest.mark.parametrize("case", MANY)
def test_expert_matvec_of_many_entries(dev, case):
    t, e, k, n, K, drop, per, swiglu = case
    assert _many(t, e, k, n, swiglu)
    rng = np.random.default_rng(t * n + K)
    ids, weight = _ids(rng, t, e, k, drop), _weights(rng, e, n, K)
    xb = _bits(rng.standard_normal((t, k, K) if per else (t, K)))
    print(f"many entries {case}", flush=True)
    xd, wd = bf16_dev(xb, dev), torch.from_numpy(weight).to(dev)
    got = mtb.ep_nvfp4_expert_matvec(xd, wd, torch.from_numpy(ids).to(dev), swiglu=swiglu)
    _check_matvec(got, expert.f64(xb), weight, ids, swiglu, f"many entries {case}")
    assert not host(got)[ids < 0].any()
    again = mtb.ep_nvfp4_expert_matvec(xd, wd, torch.from_numpy(ids.astype(np.int64)).to(dev), swiglu=swiglu)
    assert_bytes_equal(host(again), host(got), "the same call with 64-bit ids")


@pytest.mark.parametrize("idt", [np.int32, np.int64])
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_entries_with_bad_ids(dev, idt, swiglu):
    t, e, k, n, K = 150, 16, 2, 2022, 128
    assert _many(t, e, k, n, swiglu)
    rng = np.random.default_rng(5)
    ids, weight = _ids(rng, t, e, k, 0.05).astype(idt), _weights(rng, e, n, K)
    good = ids.copy()
    bad = [(0, 0, e), (17, 1, -2), (t - 1, 1, 2 ** 31 - 1 if idt is np.int32 else 2 ** 33)]
    for i, j, v in bad:
        ids[i, j], good[i, j] = v, -1
    x = rng.standard_normal((t, K)).astype(np.float32)
    xb = _bits(x)
    xd, wd, err = bf16_dev(xb, dev), torch.from_numpy(weight).to(dev), torch.zeros(1, dtype=torch.int32, device=dev)
    got = mtb.ep_nvfp4_expert_matvec(xd, wd, torch.from_numpy(ids).to(dev), swiglu=swiglu, d_error=err)
    assert int(err.item()) == mtb.EP_DEVERR_EXPERT_ID
    _check_matvec(got, expert.f64(xb), weight, good, swiglu, "bad ids")
    assert not host(got)[good < 0].any()
    err.zero_()
    again = mtb.ep_nvfp4_expert_matvec(xd, wd, torch.from_numpy(good).to(dev), swiglu=swiglu, d_error=err)
    assert int(err.item()) == 0
    assert_bytes_equal(host(again), host(got), "the same call with the ids marked")


@pytest.mark.parametrize("t", [16, 17, 70])
@pytest.mark.parametrize("n,K,swiglu", [(32700, 64, False), (32660, 192, True)])
def test_dense_matvec_of_many_rows(dev, t, n, K, swiglu):
    assert _many(t, 1, 1, n, swiglu)
    rng = np.random.default_rng(n + t)
    weight = _weights(rng, 1, n, K)[0]
    xb = _bits(rng.standard_normal((t, K)))
    print(f"dense, many rows {t} {n} {K}", flush=True)
    got = mtb.ep_nvfp4_expert_matvec(bf16_dev(xb, dev), torch.from_numpy(weight).to(dev), swiglu=swiglu)
    _check_matvec(got, expert.f64(xb), weight, None, swiglu, "dense, many rows")


def test_many_entries_keep_special_values_in_their_row(dev):
    t, e, k, n, K = 150, 16, 2, 2022, 128
    rng = np.random.default_rng(6)
    ids, weight = _ids(rng, t, e, k, 0.05), _weights(rng, e, n, K)
    x = rng.standard_normal((t, K)).astype(np.float32)
    clean = x.copy()
    x[3, 5], x[40, 0] = np.nan, np.inf
    clean[3], clean[40] = 0, 0
    got = host(mtb.ep_nvfp4_expert_matvec(bf16_dev(_bits(x), dev), torch.from_numpy(weight).to(dev),
                                          torch.from_numpy(ids).to(dev)))
    keep = np.ones(t, dtype=bool)
    keep[[3, 40]] = False
    assert np.isnan(expert.f64(got)[3][ids[3] >= 0]).all()
    _check_matvec(got[keep], expert.f64(_bits(clean))[keep], weight, ids[keep], False, "other rows")
