"""The linear part of a quantized decoder block on the library's operators.

    python examples/decoder_block.py [--tokens 8] [--check]

A block receives the output of its attention and the residual stream:

    r, q, s = norm_gate_residual(attention, residual, w1, quantize=True)   norm + residual, 8-bit codes
    p       = gemm_w8a8(q, s, W, W_scales)                                 an 8-bit projection of them
    r, h    = norm_gate_residual(p, r, w3, post_weight=w2, gate=g,         norm after it, gate, scaled
                                 residual_scale=a)                         residual, norm before the MLP
    m       = moe(h, router, gate, up, down, ...)                          experts in packed int4
    r, h    = norm_gate_residual(m, r, w5, post_weight=w4)                 into the next block

Weights are random: the projection is quantized by quantize_rows (one scale for
each output channel), the experts by quantize_pack.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import weight_only_quantization_pack_amd as awq  # noqa: E402


class Block:
    def __init__(self, width=1024, inter=512, experts=16, top_k=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device=device)

        self.width, self.inter, self.experts, self.top_k = width, inter, experts, top_k
        self.proj = (randn(width, width) * width ** -0.5).half()
        self.proj_q, self.proj_scales = awq.quantize_rows(self.proj)
        self.router = (2.0 * width ** -0.5 * randn(experts, width)).half()
        self.norms = [(1.0 + 0.1 * randn(width)).half() for _ in range(5)]
        self.gate = torch.tanh(randn(width)).half()
        self.residual_scale = 0.9

        def packed(rows, cols):
            layers = [awq.quantize_pack((cols ** -0.5 * randn(rows, cols)).half()) for _ in range(experts)]
            return tuple(torch.stack(t) for t in zip(*layers))

        self.gate_proj, self.up_proj, self.down_proj = (packed(inter, width), packed(inter, width),
                                                        packed(width, inter))

    def __call__(self, attention, residual):
        """(residual stream, normed input of the next block) of fp16 [T][width], T <= 64."""
        r, q, s = awq.norm_gate_residual(attention, residual, self.norms[0], quantize=True)
        p = awq.gemm_w8a8(q, s, self.proj_q, self.proj_scales)
        r, h = awq.norm_gate_residual(p, r, self.norms[2], post_weight=self.norms[1], gate=self.gate,
                                      residual_scale=self.residual_scale)
        m = awq.moe(h, self.router, self.gate_proj, self.up_proj, self.down_proj, inter=self.inter,
                    top_k=self.top_k)
        return awq.norm_gate_residual(m, r, self.norms[4], post_weight=self.norms[3])

    def plain(self, attention, residual):
        """The same block in 64 bits on the dequantized weights, with the roundings that storage makes."""
        def norm(v, w):
            return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w.double()

        def unpacked(layer, rows, cols):
            return torch.stack([awq.fake_quantize(*(t[e].contiguous() for t in layer), N=rows, K=cols)
                                for e in range(self.experts)]).double()

        w1, w2, w3, w4, w5 = self.norms
        r = residual.double() + attention.double()
        h = norm(r, w1)
        r = r.half().double()
        scale = h.abs().amax(-1, keepdim=True) / 127.0
        p = (torch.round(h / scale) @ self.proj_q.double().t()) * scale * self.proj_scales.double()
        r = self.residual_scale * r + self.gate.double() * norm(p.half().double(), w2)
        x = norm(r, w3).half().double()
        r = r.half().double()
        logits = x @ self.router.double().t()
        top = torch.sort(logits, dim=-1, descending=True, stable=True)
        ids, weight = top.indices[:, :self.top_k], torch.softmax(top.values[:, :self.top_k], dim=-1)
        gate, up, down = (unpacked(self.gate_proj, self.inter, self.width), unpacked(self.up_proj, self.inter, self.width),
                          unpacked(self.down_proj, self.width, self.inter))
        m = torch.zeros_like(x)
        for t in range(x.shape[0]):
            for e, w in zip(ids[t].tolist(), weight[t]):
                a = gate[e] @ x[t]
                m[t] += w * (down[e] @ (a * torch.sigmoid(a) * (up[e] @ x[t])))
        r = r + norm(m.half().double(), w4)
        return r, norm(r, w5)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=8, help="tokens of the decode batch (at most 64)")
    ap.add_argument("--check", action="store_true", help="compare with the block in 64 bits")
    a = ap.parse_args(argv)
    block = Block()
    g = torch.Generator(device="cuda").manual_seed(1)
    attention, residual = (torch.randn(a.tokens, block.width, generator=g, device="cuda").half() for _ in range(2))
    r, h = block(attention, residual)
    print(f"block of {a.tokens} tokens: residual {tuple(r.shape)} {r.dtype}, next input {tuple(h.shape)} {h.dtype}")
    if not a.check:
        return 0.0
    worst = max(float((x.double() - y).norm() / y.norm()) for x, y in zip((r, h), block.plain(attention, residual)))
    print(f"relative difference from the block in 64 bits: {worst:.2e}")
    return worst


if __name__ == "__main__":
    sys.exit(1 if main() > 5e-3 else 0)
