"""Timed cases of an expert layer's products and of the norm in front of it.

Three groups, as one layer uses them:

* products of grouped BF16 rows with their experts' weights:
  ``ep_bf16_grouped_gemm`` (the forward product), ``ep_bf16_grouped_dgrad`` (the
  rows' gradient) and ``ep_bf16_grouped_wgrad`` (the weights' gradient);
* microscaled 4-bit values (E2M1 codes, a power of two per 32):
  ``ep_mxfp4_pack`` and ``ep_mxfp4_unpack``, and ``ep_mxfp4_grouped_gemm``, the
  product of MXFP4 or MXFP8 rows with MXFP4 weights;
* ``rmsnorm_mxfp8``, the root-mean-square norm after the residual's addition
  with an MXFP8 output, and its gradient ``drmsnorm``.

``run`` computes a case in plain torch operations in 32 bits, or by the
package's kernels where ``own`` is true; ``exact`` gives the same outputs from
the definitions in 64 bits.
"""

import math

import torch

own = False

ALIGN = 16  # grouped rows of one expert start at multiples of this
EPS = 1e-6


def _dev():
    return torch.device("cuda")


# ------------------------------------------------------------------ the cases
def listed():
    rt = dict(skew=0.0, unused=0.0)
    return [
        # one token of a chat through its experts' gate and up projections: latency
        dict(rt, op="gemm", name="gemm_1x4096_e8_top2_4096", tokens=1, k=4096, n=4096, experts=8, top_k=2),
        # a ragged batch at odd widths, some slots dropped
        dict(rt, op="gemm", name="gemm_1037x1001_e7_top3_515", tokens=1037, k=1001, n=515, experts=7, top_k=3, unused=0.2),
        # the largest forward: a long prompt through the gate and up projections
        dict(rt, op="gemm", name="gemm_16384x7168_e32_top8_4096", tokens=16384, k=7168, n=4096, experts=32, top_k=8),
        # a training micro-batch's rows' gradient, experts unevenly loaded
        dict(rt, op="dgrad", name="dgrad_4096x4096_e8_top2_4096", tokens=4096, k=4096, n=4096, experts=8, top_k=2, skew=1.2),
        # a training batch's weight gradient
        dict(rt, op="wgrad", name="wgrad_32768x4096_e16_top2_4096", tokens=32768, k=4096, n=4096, experts=16, top_k=2,
             f32=False),
        # activations or weights to 4 bits and back
        dict(op="pack", name="pack_16384x7168", tokens=16384, k=7168),
        # one token through its experts' down projections in 4 bits: latency
        dict(rt, op="mx", name="mx4_1x2048_e8_top2_4096", tokens=1, k=2048, n=4096, experts=8, top_k=2, eight=False),
        # a ragged batch of 8-bit rows with 4-bit weights, some slots dropped
        dict(rt, op="mx", name="mx8_1037x4096_e8_top2_4096", tokens=1037, k=4096, n=4096, experts=8, top_k=2, eight=True,
             unused=0.1),
        # a long prompt through the gate and up projections in 4 bits
        dict(rt, op="mx", name="mx4_16384x7168_e32_top8_4096", tokens=16384, k=7168, n=4096, experts=32, top_k=8,
             eight=False),
        # the norm in front of the layer: one token (latency) and a long prompt
        dict(op="norm", name="norm_1x4096", tokens=1, k=4096, residual=True),
        dict(op="norm", name="norm_16384x7168", tokens=16384, k=7168, residual=True),
        # its gradient for a training batch
        dict(op="dnorm", name="dnorm_14841x4096", tokens=14841, k=4096, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "dgrad", "wgrad", "mx", "mx", "pack", "norm", "dnorm"])
    tokens = _log(rng, 1, 16384)
    if op in ("pack", "norm", "dnorm"):
        case = dict(op=op, tokens=tokens, k=32 * _log(rng, 2, 224))
        return case if op == "pack" else dict(case, residual=rng.random() < 0.7)
    e = rng.choice([2, 5, 8, 16, 32])
    case = dict(op=op, tokens=tokens, n=_log(rng, 16, 4096), experts=e, top_k=rng.randint(1, min(e, 8)),
                unused=rng.choice([0.0, 0.0, 0.05, 0.3]))
    if op == "mx":
        case.update(k=32 * _log(rng, 2, 224), eight=rng.random() < 0.5)
    else:
        case.update(k=_log(rng, 64, 7168))
        if rng.random() < 0.7:
            case.update(k=case["k"] // 8 * 8, n=max(8, case["n"] // 8 * 8))
        if op == "wgrad":
            case.update(f32=rng.random() < 0.5)
    # the plain form pads every expert to the fullest: uneven loads at moderate sizes only
    small = e * tokens * (case["k"] + case["n"]) <= 1 << 30
    return dict(case, skew=rng.choice([0.0, 1.2]) if small else 0.0)


# ------------------------------------------------------------------ inputs
def _routing(g, case):
    """The expert of every slot (distinct ones for a token), -1 for dropped slots."""
    dev = _dev()
    tokens, experts = case["tokens"], case["experts"]
    logits = torch.randn(tokens, experts, generator=g, device=dev)
    logits -= case["skew"] * torch.log1p(torch.arange(experts, device=dev, dtype=torch.float32))
    ids = torch.topk(logits, case["top_k"], dim=1).indices.to(torch.int32)
    return ids.masked_fill(torch.rand(ids.shape, generator=g, device=dev) < case["unused"], -1).contiguous()


def _plan(ids, experts):
    """The routing plan of ids [T, k]: grouped rows in expert order, each expert's
    rows in token order and padded to a multiple of ALIGN."""
    dev = ids.device
    tokens, top_k = ids.shape
    flat = ids.reshape(-1).long()
    n = flat.numel()
    counts = torch.bincount(flat[flat >= 0], minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=dev)
    offsets[1:] = torch.cumsum((counts + ALIGN - 1) // ALIGN * ALIGN, 0)
    first = torch.cumsum(counts, 0) - counts
    order = torch.argsort(torch.where(flat >= 0, flat, torch.full_like(flat, experts)), stable=True)
    used = int((flat >= 0).sum())
    order = order[:used]
    row = offsets[flat[order]] + torch.arange(used, device=dev) - first[flat[order]]
    r_cap = n + experts * (ALIGN - 1)
    dst = torch.full((n,), -1, dtype=torch.int32, device=dev)
    src = torch.full((r_cap,), -1, dtype=torch.int32, device=dev)
    dst[order] = row.to(torch.int32)
    src[row] = (order // top_k).to(torch.int32)
    return dict(counts=counts.to(torch.int32), offsets=offsets.to(torch.int32), dst_row=dst.view(tokens, top_k),
                src_row=src, r_cap=r_cap, num_experts=experts, alignment=ALIGN)


def _grouped(g, plan, width, scale=1.0):
    """BF16 grouped rows as the dispatch leaves them: padding rows zero."""
    rows = torch.randn(plan["r_cap"], width, generator=g, device=_dev(), dtype=torch.bfloat16)
    return rows.mul_(scale).masked_fill_((plan["src_row"] < 0)[:, None], 0.0)


def _pow2(e):
    """2^e in FP32 for whole e in [-127, 127], from the bits (a power function may round)."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).view(torch.float32)


def _block_exponent(amax, mantissa, bits):
    """The least e with amax <= (mantissa * 2^bits) * 2^e, mantissa in [0.5, 1); 0 for
    amax 0; within [-127, 127]."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [0.5, 1)
    e = torch.where(m > mantissa, e - bits + 1, e - bits)
    return torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))


def _mxfp4_exponent(amax):
    return _block_exponent(amax, 0.75, 3)  # 6 = 0.75 * 2^3


def _mxfp8_exponent(amax):
    return _block_exponent(amax, 0.875, 9)  # 448 = 0.875 * 2^9


def _e2m1_round(v):
    """Values of magnitude at most 6 onto the grid 0, .5, 1, 1.5, 2, 3, 4, 6, ties to even."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v)


def _mxfp4(x):
    """FP32 rows [n, k] -> (codes uint8 [n, k/2], even element in the low nibble; scales uint8 [n, k/32])."""
    n, k = x.shape
    blocks = x.view(n, k // 32, 32)
    e = _mxfp4_exponent(blocks.abs().amax(2))
    v = _e2m1_round(blocks * _pow2(-e)[:, :, None]).view(n, k // 2, 2)
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code |= torch.signbit(v).to(torch.uint8) << 3
    return code[:, :, 0] | (code[:, :, 1] << 4), (e + 127).to(torch.uint8)


def _mxfp8(x):
    """FP32 rows [n, k] -> (E4M3 bytes [n, k], scales uint8 [n, k/32])."""
    n, k = x.shape
    blocks = x.view(n, k // 32, 32)
    e = _mxfp8_exponent(blocks.abs().amax(2))
    q = (blocks * _pow2(-e)[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(n, k), (e + 127).to(torch.uint8)


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(seed)
    op, t, k = case["op"], case["tokens"], case["k"]
    if op in ("pack", "norm", "dnorm"):
        # rows of different size, a few large values
        x = torch.randn(t, k, generator=g, device=dev) * torch.exp(torch.randn(t, 1, generator=g, device=dev))
        x = (x * torch.where(torch.rand(t, k, generator=g, device=dev) < 1e-3, 20.0, 1.0)).to(torch.bfloat16)
        state = dict(case=case, x=x)
        if op == "pack":
            return state
        state["weight"] = (1 + 0.2 * torch.randn(k, generator=g, device=dev)).to(torch.bfloat16)
        other = None
        if case["residual"]:
            other = torch.randn(t, k, generator=g, device=dev).to(torch.bfloat16)
        if op == "norm":
            return dict(state, residual=other)
        state["rstd"] = torch.rsqrt(x.float().square().mean(1) + EPS)
        state["dy"] = (1e-2 * torch.randn(t, k, generator=g, device=dev)).to(torch.bfloat16)
        return dict(state, dh=None if other is None else other.mul_(1e-2))
    e, n = case["experts"], case["n"]
    plan = _plan(_routing(g, case), e)
    state = dict(case=case, plan=plan, most=int(plan["counts"].max()))
    if op == "mx":
        rows = _grouped(g, plan, k).float()
        state["data"], state["scales"] = _mxfp8(rows) if case["eight"] else _mxfp4(rows)
        codes = torch.empty(e, n, k // 2, dtype=torch.uint8, device=dev)
        scales = torch.empty(e, n, k // 32, dtype=torch.uint8, device=dev)
        for i in range(e):
            codes[i], scales[i] = _mxfp4(torch.randn(n, k, generator=g, device=dev) / math.sqrt(k))
        return dict(state, wcodes=codes, wscales=scales)
    if op != "wgrad":
        state["weight"] = torch.randn(e, n, k, generator=g, device=dev, dtype=torch.bfloat16).div_(math.sqrt(k))
    if op != "dgrad":
        state["rows"] = _grouped(g, plan, k)
    if op != "gemm":
        state["dout"] = _grouped(g, plan, n, 1e-2)
    return state


# ------------------------------------------------------------------ the plain forms
def _by_expert(plan, most, rows):
    """Grouped rows [r_cap, w] -> FP32 [E, most, w], zeros past each expert's count; and where they came from."""
    i = torch.arange(most, device=rows.device)
    used = i < plan["counts"][:, None]
    at = torch.where(used, plan["offsets"][:-1, None] + i, 0).long()
    return torch.where(used[:, :, None], rows[at].float(), 0.0), at, used


def _back(plan, y, at, used):
    """FP32 [E, most, w] -> BF16 grouped rows, the others zero."""
    out = torch.zeros(plan["r_cap"], y.shape[2], dtype=torch.bfloat16, device=y.device)
    out[at[used]] = y[used].to(torch.bfloat16)
    return out


def _product(s, rows, weight):
    """Each expert's rows times its weight^T; weight: experts (None: all) -> FP32 [., n, k]."""
    plan, c = s["plan"], s["case"]
    if c["tokens"] * c["top_k"] <= c["experts"]:  # few rows: only their experts' weights are read
        dst = plan["dst_row"].reshape(-1)
        at = dst.clamp(min=0).long()
        e = (torch.searchsorted(plan["offsets"], dst.clamp(min=0), right=True) - 1).clamp(max=c["experts"] - 1)
        y = (weight(e) @ rows[at].float()[:, :, None])[:, :, 0]
        out = torch.zeros(plan["r_cap"], y.shape[1], dtype=torch.bfloat16, device=y.device)
        out[dst[dst >= 0].long()] = y[dst >= 0].to(torch.bfloat16)
        return out
    x, at, used = _by_expert(plan, s["most"], rows)
    return _back(plan, x @ weight(None).transpose(1, 2), at, used)


def _e4m3(b):
    """E4M3 bytes -> FP32, from the bits."""
    b = b.to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).float()
    v = torch.where(e > 0, (8.0 + m) * _pow2(e - 10), m * 2.0 ** -9)
    return torch.where(b >= 128, -v, v)


def _scaled(v, scales):
    """Values [.., k] times the powers of two of their blocks of 32."""
    shape = v.shape
    return (v.view(*shape[:-1], shape[-1] // 32, 32) * _pow2(scales.int() - 127)[..., None]).view(shape)


def _mxfp4_values(codes, scales):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat([grid, -grid])
    c = codes.int()
    v = torch.stack([grid[c & 15], grid[c >> 4]], -1)
    return _scaled(v.view(*codes.shape[:-1], 2 * codes.shape[-1]), scales)


def _plain_norm(s):
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(torch.bfloat16)
    v = h.float()
    rstd = torch.rsqrt(v.square().mean(1) + EPS)
    y = v * rstd[:, None] * s["weight"].float()
    t, k = y.shape
    blocks = y.view(t, k // 32, 32)
    e = _mxfp8_exponent(blocks.abs().amax(2))[:, :, None]
    q = (blocks * _pow2(-e)).to(torch.float8_e4m3fn).float() * _pow2(e)
    return {"h": h, "rstd": rstd, "y": q.view(t, k).to(torch.bfloat16)}


def _plain_dnorm(s):
    h, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = r * (g - h * (r * r * (g * h).mean(1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(torch.bfloat16), "dweight": (dy * (h * r)).sum(0)}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import moe_token_block_amd as m

        if op == "gemm":
            return m.ep_bf16_grouped_gemm(state["rows"], state["weight"], state["plan"])
        if op == "dgrad":
            return m.ep_bf16_grouped_dgrad(state["dout"], state["weight"], state["plan"])
        if op == "wgrad":
            return m.ep_bf16_grouped_wgrad(state["dout"], state["rows"], state["plan"],
                                           dtype=torch.float32 if case["f32"] else torch.bfloat16)
        if op == "mx":
            return m.ep_mxfp4_grouped_gemm(state["data"], state["scales"], state["wcodes"], state["wscales"], state["plan"])
        if op == "pack":
            return m.ep_mxfp4_unpack(*m.ep_mxfp4_pack(state["x"]))
        if op == "norm":
            data, scales, h, rstd = m.rmsnorm_mxfp8(state["x"], state["weight"], state["residual"], eps=EPS)
            return {"h": h, "rstd": rstd, "y": m.ep_mxfp8_unpack(data, scales)}
        dx, dweight = m.drmsnorm(state["dy"], state["x"], state["weight"], state["rstd"], state["dh"])
        return {"dx": dx, "dweight": dweight}

    if op == "gemm":
        w = state["weight"]
        return _product(state, state["rows"], lambda e: (w if e is None else w[e]).float())
    if op == "dgrad":
        w = state["weight"]
        return _product(state, state["dout"], lambda e: (w if e is None else w[e]).float().transpose(1, 2))
    if op == "wgrad":
        d, _, _ = _by_expert(state["plan"], state["most"], state["dout"])
        x, _, _ = _by_expert(state["plan"], state["most"], state["rows"])
        return (d.transpose(1, 2) @ x).to(torch.float32 if case["f32"] else torch.bfloat16)
    if op == "mx":
        if case["eight"]:
            rows = _scaled(_e4m3(state["data"]), state["scales"])
        else:
            rows = _mxfp4_values(state["data"], state["scales"])
        c, s = state["wcodes"], state["wscales"]
        return _product(state, rows, lambda e: _mxfp4_values(c, s) if e is None else _mxfp4_values(c[e], s[e]))
    if op == "pack":
        x = state["x"].float()
        blocks = x.view(x.shape[0], -1, 32)
        e = _mxfp4_exponent(blocks.abs().amax(2))[:, :, None]
        return (_e2m1_round(blocks * _pow2(-e)) * _pow2(e)).view(x.shape).to(torch.bfloat16)
    return _plain_norm(state) if op == "norm" else _plain_dnorm(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, t, k = case["op"], case["tokens"], case["k"]
    if op == "pack":  # the values in, the 4 bits out; the 4 bits in, their values out
        return {"bytes": t * k * (2.0 + 2 * (1 / 2 + 1 / 32) + 2), "flops": 3.0 * t * k}
    if op == "norm":  # as above with 8 bits, the sum written beside them
        return {"bytes": t * k * (2.0 + (2 if case["residual"] else 0) + 2 + 2 * (1 + 1 / 32) + 2) + 2 * k + 4 * t,
                "flops": 6.0 * t * k}
    if op == "dnorm":
        return {"bytes": t * k * (6.0 + (2 if case["residual"] else 0)) + 6 * k + 4 * t, "flops": 10.0 * t * k}
    e, n, top = case["experts"], case["n"], case["top_k"]
    entries = t * top * (1 - case["unused"])
    used = e * (1 - (1 - entries / t / e) ** t)  # experts that some token names
    r_cap = t * top + e * (ALIGN - 1)
    flops = 2.0 * entries * n * k
    if op == "gemm":
        return {"bytes": 2 * (entries * k + used * n * k + r_cap * n), "flops": flops}
    if op == "dgrad":
        return {"bytes": 2 * (entries * n + used * n * k + r_cap * k), "flops": flops}
    if op == "wgrad":
        return {"bytes": 2 * entries * (n + k) + (4 if case["f32"] else 2) * e * n * k, "flops": flops}
    four = 1 / 2 + 1 / 32
    return {"bytes": entries * k * (1 + 1 / 32 if case["eight"] else four) + used * n * k * four + 2 * r_cap * n,
            "flops": flops}


# ------------------------------------------------------------------ in 64 bits
def _two(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_mx(bytes_, scales, four):
    """Codes and block scales -> values in 64 bits, by the formats' fields."""
    if four:
        c = torch.stack([bytes_ & 15, bytes_ >> 4], -1).reshape(*bytes_.shape[:-1], -1).long()
        e, m, neg, bias, frac = (c >> 1) & 3, c & 1, c >= 8, 1, 1
    else:
        c = bytes_.long()
        e, m, neg, bias, frac = (c >> 3) & 15, c & 7, c >= 128, 7, 3
    lead = torch.where(e > 0, 1.0, 0.0).double()
    v = (lead + m.double() / 2 ** frac) * _two(e.clamp(min=1) - bias)
    return torch.where(neg, -v, v) * _two(scales.long() - 127).repeat_interleave(32, -1)


def _exact_round(u, bits, low):
    """To `bits` mantissa bits below the leading one, none below 2^low."""
    step = _two(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** (low + bits)))) - bits)
    return torch.round(u / step) * step


def _exact_blocks(y, largest, bits, low):
    q = y.reshape(-1, 32)
    top = q.abs().amax(1, keepdim=True)
    e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / largest)), 0.0)
    return (_exact_round(q * _two(-e), bits, low) * _two(e)).view_as(y)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "pack":
        return _exact_blocks(s["x"].double(), 6.0, 1, -1)
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            # FP32 holds the sum of two BF16 numbers of like size exactly or rounds it once; the value is BF16's nearest
            h = (s["x"].float() + s["residual"].float()).to(torch.bfloat16).double()
        rstd = 1 / torch.sqrt((h * h).sum(1) / case["k"] + EPS)
        y = h * rstd[:, None] * s["weight"].double()
        return {"h": h, "rstd": rstd, "y": _exact_blocks(y, 448.0, 3, -9)}
    if op == "dnorm":
        h, dy, r = s["x"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        xhat, g = h * r, dy * s["weight"].double()
        dx = r * (g - xhat * ((g * xhat).sum(1, keepdim=True) / case["k"]))
        return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dweight": (dy * xhat).sum(0)}
    plan = s["plan"]
    lo, cnt = plan["offsets"].tolist(), plan["counts"].tolist()
    spans = [(i, slice(lo[i], lo[i] + cnt[i])) for i in range(case["experts"])]
    if op == "wgrad":
        out = torch.zeros(case["experts"], case["n"], case["k"], dtype=torch.float64, device=_dev())
        for i, at in spans:
            out[i] = s["dout"][at].double().T @ s["rows"][at].double()
        return out
    out = torch.zeros(plan["r_cap"], case["k"] if op == "dgrad" else case["n"], dtype=torch.float64, device=_dev())
    for i, at in spans:
        if cnt[i] == 0:
            continue
        if op == "gemm":
            out[at] = s["rows"][at].double() @ s["weight"][i].double().T
        elif op == "dgrad":
            out[at] = s["dout"][at].double() @ s["weight"][i].double()
        else:
            x = _exact_mx(s["data"][at], s["scales"][at], not case["eight"])
            out[at] = x @ _exact_mx(s["wcodes"][i], s["wscales"][i], True).T
    return out
