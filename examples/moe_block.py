"""One mixture-of-experts block on the library: router, routed experts on 8-bit weights,
shared expert on bf16 weights, and an 8-bit projection of the result.

    logits       = x Wr^T                                  shared_mlp_linear (bf16)
    ids, weights = route(logits)                           shared_mlp_route
    routed       = sum_j weights_j expert_{ids_j}(x)       shared_mlp_experts_fp8
    shared       = down(SiLU(x Wg^T) * (x Wu^T))           shared_mlp_forward (bf16)
    y            = (routed + shared) Wl^T                  shared_mlp_linear_fp8

    python examples/moe_block.py [--tokens 16] [--hidden 7168] [--inter 768] [--experts 64] [--steps 20]

Seeded random weights; prints the time of a step and how far the block is from the same
formulas computed with torch in fp32 from the 8-bit weights' values.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_shared_expert_amd import binding  # noqa: E402


class Block:
    """Weights of one block on the GPU, in the forms the calls take."""

    def __init__(self, hidden, inter, experts, topk, latent, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def w(*shape):
            return torch.randn(*shape, generator=g, device=device) / shape[-1] ** 0.5

        self.topk, self.inter = topk, inter
        self.router = w(experts, hidden).bfloat16()
        self.bias = 0.05 * torch.randn(experts, generator=g, device=device)
        gate_up, s = binding.quantize_fp8(w(2 * experts, inter, hidden), 128)  # gate and up halves quantised apart
        self.gate_up = gate_up.view(experts, 2 * inter, hidden)
        self.s_gate_up = s.view(experts, -1, s.shape[-1])
        self.down, self.s_down = binding.quantize_fp8(w(experts, hidden, inter), 128)
        self.shared_gate_up, self.shared_down = w(2 * inter, hidden).bfloat16(), w(hidden, inter).bfloat16()
        self.latent, self.s_latent = binding.quantize_fp8(w(latent, hidden), 128)

    def __call__(self, x):
        logits = torch.empty(x.shape[0], self.router.shape[0], dtype=torch.float32, device=x.device)
        binding.shared_mlp_linear(x, self.router, logits)
        ids, weights = binding.route(logits, self.topk, bias=self.bias)
        out = binding.experts_fp8(x, ids, weights, self.gate_up, self.s_gate_up, self.down, self.s_down)
        out += binding.forward(x, self.shared_gate_up, self.shared_down)
        return binding.linear_fp8(out, self.latent, self.s_latent)

    def plain(self, x):
        """The same block in torch, fp32, expert by expert."""
        def rows(v):
            q, s = binding.quantize_fp8(v)
            return q.float() * s.repeat_interleave(128, 1)[:, :v.shape[1]]

        def blocks(q, s):
            return q.float() * s.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]

        logits = x.float() @ self.router.float().t()
        score = torch.sigmoid(logits)
        ids = torch.sort(score + self.bias, dim=1, descending=True, stable=True)[1][:, :self.topk]
        weights = score.gather(1, ids)
        weights = weights / weights.sum(1, keepdim=True)
        xq, out, n = rows(x), torch.zeros(x.shape, device=x.device), self.s_gate_up.shape[1] // 2
        for e in range(self.router.shape[0]):
            t, j = (ids == e).nonzero(as_tuple=True)
            if t.numel():
                g = xq[t] @ blocks(self.gate_up[e, :self.inter], self.s_gate_up[e, :n]).t()
                u = xq[t] @ blocks(self.gate_up[e, self.inter:], self.s_gate_up[e, n:]).t()
                y = rows(torch.nn.functional.silu(g) * u) @ blocks(self.down[e], self.s_down[e]).t()
                out.index_add_(0, t, y * weights[t, j, None])
        gu = x.float() @ self.shared_gate_up.float().t()
        h = torch.nn.functional.silu(gu[:, :self.inter]) * gu[:, self.inter:]
        out = out.bfloat16() + (h @ self.shared_down.float().t()).bfloat16()
        return rows(out) @ blocks(self.latent, self.s_latent).t()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 16), ("hidden", 7168), ("inter", 768), ("experts", 64), ("topk", 8), ("latent", 2112),
                        ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    block = Block(a.hidden, a.inter, a.experts, a.topk, a.latent)
    x = torch.randn(a.tokens, a.hidden, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    y, ref = block(x).float(), block.plain(x)
    off = ((y - ref).norm() / ref.norm()).item()
    for _ in range(3):
        block(x)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        block(x)
    torch.cuda.synchronize()
    us = (time.perf_counter() - t) / a.steps * 1e6
    print(f"{a.tokens} tokens, {a.experts} experts of {a.inter}, top {a.topk}: {us:.1f} us a step, {off:.2e} off the plain form")
    return off


if __name__ == "__main__":
    main()
