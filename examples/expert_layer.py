"""One expert layer on the package's calls: a training step whose activations are
kept in 8 bits, prompts served from 4-bit weights and 8-bit rows, and single tokens
from 4-bit weights.

    python examples/expert_layer.py [--tokens 4096] [--hidden 4096] [--ffn 2048] [--experts 8] [--top-k 2]

Training: route plan -> BF16 dispatch -> gate/up product -> SwiGLU with its
pre-activation kept as MXFP8 -> down product -> weighted combine, and back.  A
block adds the residual and the norm in front (``block_forward``,
``block_backward``).  Prompts: the norm's MXFP8 rows to their experts, products with
MXFP4 weights.  Single tokens: the weights as NVFP4 rows, each token's rows by
``ep_nvfp4_expert_matvec`` and the combine.  Nothing waits for the host, so that each
of them can be captured in a graph.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_token_block_amd as m  # noqa: E402


class ExpertLayer:
    """w1 [E, 2F, H] (gate and up halves), w2 [E, H, F], BF16."""

    def __init__(self, experts, hidden, ffn, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.w1 = (rand(experts, 2 * ffn, hidden) / hidden ** 0.5).bfloat16()
        self.w2 = (rand(experts, hidden, ffn) / ffn ** 0.5).bfloat16()

    # -------------------------------------------------------------- training
    def forward(self, x, topk_idx, weights):
        """Output [T, H] and what the backward pass needs: no BF16 pre-activation
        and no SwiGLU output among it."""
        plan = m.ep_route_plan(topk_idx, self.w1.shape[0])
        rows = m.ep_bf16_dispatch(x, plan)
        act, data, scales = m.swiglu_mxfp8_checkpoint(m.ep_bf16_grouped_gemm(rows, self.w1, plan))
        y = m.ep_bf16_grouped_gemm(act, self.w2, plan)
        return m.ep_bf16_combine(y, plan, weights), (plan, rows, data, scales, y, weights)

    def backward(self, dout, kept):
        """Gradients of x, the router weights, w1 and w2."""
        plan, rows, data, scales, y, weights = kept
        dy, dweights = m.ep_bf16_combine_bwd(dout, y, plan, weights)
        dact = m.ep_bf16_grouped_dgrad(dy, self.w2, plan)
        dpre, act = m.dswiglu_mxfp8_checkpoint(data, scales, dact)
        dw2 = m.ep_bf16_grouped_wgrad(dy, act, plan)
        dw1 = m.ep_bf16_grouped_wgrad(dpre, rows, plan)
        drows = m.ep_bf16_grouped_dgrad(dpre, self.w1, plan)
        return m.ep_bf16_combine(drows, plan), dweights, dw1, dw2

    # -------------------------------------------------------------- serving
    def pack(self):
        """The weights as NVFP4 rows, laid out once."""
        rows = lambda w: m.ep_nvfp4_pack(w.reshape(-1, w.shape[2])).view(w.shape[0], w.shape[1], -1)  # noqa: E731
        return rows(self.w1), rows(self.w2)

    def pack_mxfp4(self):
        """The weights as MXFP4 (codes, scales), laid out once."""
        pack = lambda w: tuple(v.view(*w.shape[:2], -1) for v in m.ep_mxfp4_pack(w.view(-1, w.shape[2])))  # noqa: E731
        return pack(self.w1), pack(self.w2)


# ------------------------------------------------------------------ with the norm in front
def block_forward(layer, x, residual, norm_weight, topk_idx, weights):
    """h = x + residual and layer(norm(h)): what the next block adds, its residual, and
    what the backward pass needs.  The experts see the 8-bit rows' values."""
    data, scales, h, rstd = m.rmsnorm_mxfp8(x, norm_weight, residual)
    out, kept = layer.forward(m.ep_mxfp8_unpack(data, scales), topk_idx, weights)
    return out, h, (kept, h, rstd)


def block_backward(layer, dout, dh, norm_weight, kept):
    """Gradients for dout and for dh, which reaches h from the blocks behind: of x and
    the residual alike, the norm's weight, the router weights, w1 and w2."""
    kept, h, rstd = kept
    dy, dweights, dw1, dw2 = layer.backward(dout, kept)
    dx, dnorm = m.drmsnorm(dy, h, norm_weight, rstd, dh)
    return dx, dnorm, dweights, dw1, dw2


# ------------------------------------------------------------------ serving
def serve_prompt(x, residual, norm_weight, topk_idx, weights, packed):
    """Output [T, H] and the sum h of a prompt: 8-bit rows, 4-bit weights (``pack_mxfp4``)."""
    w1, w2 = packed
    data, scales, h, _ = m.rmsnorm_mxfp8(x, norm_weight, residual)
    plan = m.ep_route_plan(topk_idx, w2[0].shape[0])
    rows, row_scales = m.ep_mxfp8_direct_receive(data, scales, plan)
    act, _, _ = m.swiglu_mxfp8_checkpoint(m.ep_mxfp4_grouped_gemm(rows, row_scales, *w1, plan))
    data, scales, _ = m.ep_mxfp8_pack(act)
    return m.ep_bf16_combine(m.ep_mxfp4_grouped_gemm(data, scales, *w2, plan), plan, weights), h


def serve(x, topk_idx, weights, packed, entries):
    """Output [T, H] of a few tokens; ``entries``: ``ep_entry_plan`` of the batch."""
    w1, w2 = packed
    act = m.ep_nvfp4_expert_matvec(x, w1, topk_idx, swiglu=True)
    y = m.ep_nvfp4_expert_matvec(act, w2, topk_idx)
    return m.ep_bf16_combine(y.view(-1, y.shape[2]), entries, weights, topk_idx=topk_idx, num_experts=w2.shape[0])


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 4096), ("ffn", 2048), ("experts", 8), ("top-k", 2), ("serve", 4)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    dev = torch.device("cuda:0")
    torch.manual_seed(0)
    layer = ExpertLayer(a.experts, a.hidden, a.ffn, dev)
    x = torch.randn(a.tokens, a.hidden, device=dev).bfloat16()
    top = torch.topk(torch.randn(a.tokens, a.experts, device=dev), a.top_k)
    ids, weights = top.indices.int(), torch.softmax(top.values, 1)
    dout = torch.randn_like(x)

    def timed(f, n=10):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            r = f()
        torch.cuda.synchronize()
        return r, (time.perf_counter() - t) / n * 1e3

    def step():
        out, kept = layer.forward(x, ids, weights)
        return out, kept, layer.backward(dout, kept)

    (out, kept, _), ms = timed(step)
    kept_bytes = kept[2].numel() + kept[3].numel()
    print(f"training step: {a.tokens} tokens in {ms:.3f} ms; pre-activation kept in {kept_bytes / 2**20:.1f} MiB "
          f"(BF16: {2 * kept[2].numel() / 2**20:.1f})")
    norm_weight = torch.ones(a.hidden, device=dev).bfloat16()
    mx = layer.pack_mxfp4()
    residual = torch.zeros_like(x)
    (served, _), ms = timed(lambda: serve_prompt(x, residual, norm_weight, ids, weights, mx))
    normed, _, _ = block_forward(layer, x, residual, norm_weight, ids, weights)
    rel = float((served.float() - normed.float()).norm() / normed.float().norm())
    print(f"prompt: {a.tokens} tokens in {ms:.3f} ms; 4-bit against BF16 weights: {rel:.3f} of the output's norm")
    packed = layer.pack()
    n = min(a.serve, a.tokens)
    entries = m.ep_entry_plan(n, a.top_k, dev)
    served, ms = timed(lambda: serve(x[:n], ids[:n].contiguous(), weights[:n].contiguous(), packed, entries), 50)
    rel = float((served.float() - out[:n].float()).norm() / out[:n].float().norm())
    print(f"serving: {n} tokens in {ms:.3f} ms; 4-bit against BF16 weights: {rel:.3f} of the output's norm")


if __name__ == "__main__":
    main()
