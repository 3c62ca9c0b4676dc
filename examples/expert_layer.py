"""One expert layer on the package's calls: a training step whose activations are
kept in 8 bits, and tokens served from 4-bit weights.

    python examples/expert_layer.py [--tokens 4096] [--hidden 4096] [--ffn 2048] [--experts 8] [--top-k 2]

Training: route plan -> BF16 dispatch -> gate/up product -> SwiGLU with its
pre-activation kept as MXFP8 -> down product -> weighted combine, and back.  The
products of the grouped rows are torch's.  Serving: the same weights packed to
NVFP4 rows, each token's rows by ``ep_nvfp4_expert_matvec`` and the combine.
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
    def _grouped(self, rows, plan, weight):
        """rows of each expert times weight[e]^T, in the plan's grouped layout."""
        out = rows.new_zeros(rows.shape[0], weight.shape[1])
        for e, (lo, hi) in enumerate(plan["bounds"]):
            if hi > lo:
                torch.matmul(rows[lo:hi], weight[e].T, out=out[lo:hi])
        return out

    def _grouped_grad(self, left, right, plan):
        """left_e^T right_e of each expert's rows: the weights' gradients."""
        out = left.new_zeros(len(plan["bounds"]), left.shape[1], right.shape[1])
        for e, (lo, hi) in enumerate(plan["bounds"]):
            if hi > lo:
                out[e] = left[lo:hi].T @ right[lo:hi]
        return out

    def forward(self, x, topk_idx, weights):
        """Output [T, H] and what the backward pass needs: no BF16 pre-activation
        and no SwiGLU output among it."""
        plan = m.ep_route_plan(topk_idx, self.w1.shape[0])
        offsets = plan["offsets"].tolist()
        plan["bounds"] = list(zip(offsets, offsets[1:]))
        rows = m.ep_bf16_dispatch(x, plan)
        act, data, scales = m.swiglu_mxfp8_checkpoint(self._grouped(rows, plan, self.w1))
        y = self._grouped(act, plan, self.w2)
        return m.ep_bf16_combine(y, plan, weights), (plan, rows, data, scales, y, weights)

    def backward(self, dout, kept):
        """Gradients of x, the router weights, w1 and w2."""
        plan, rows, data, scales, y, weights = kept
        dy, dweights = m.ep_bf16_combine_bwd(dout, y, plan, weights)
        dact = self._grouped(dy, plan, self.w2.transpose(1, 2).contiguous())
        dpre, act = m.dswiglu_mxfp8_checkpoint(data, scales, dact)
        dw2 = self._grouped_grad(dy, act, plan)
        dw1 = self._grouped_grad(dpre, rows, plan)
        drows = self._grouped(dpre, plan, self.w1.transpose(1, 2).contiguous())
        return m.ep_bf16_combine(drows, plan), dweights, dw1, dw2

    # -------------------------------------------------------------- serving
    def pack(self):
        """The weights as NVFP4 rows, laid out once."""
        rows = lambda w: m.ep_nvfp4_pack(w.reshape(-1, w.shape[2])).view(w.shape[0], w.shape[1], -1)  # noqa: E731
        return rows(self.w1), rows(self.w2)


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
    packed = layer.pack()
    n = min(a.serve, a.tokens)
    entries = m.ep_entry_plan(n, a.top_k, dev)
    served, ms = timed(lambda: serve(x[:n], ids[:n].contiguous(), weights[:n].contiguous(), packed, entries), 50)
    rel = float((served.float() - out[:n].float()).norm() / out[:n].float().norm())
    print(f"serving: {n} tokens in {ms:.3f} ms; 4-bit against BF16 weights: {rel:.3f} of the output's norm")


if __name__ == "__main__":
    main()
