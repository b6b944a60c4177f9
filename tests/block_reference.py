"""Plain 64-bit forms of the operators beside the packed products, on numpy
arrays: what the GPU results are held against."""
import numpy as np


def to_f64(t):
    """A torch tensor (any type, either device) as float64 numpy."""
    import torch
    return t.detach().to("cpu", torch.float64).numpy()


def norm(v, weight, bias, kind, eps):
    if kind == "layer":
        v = v - v.mean(-1, keepdims=True)
    v = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * weight
    return v if bias is None else v + bias


def norm_gate_residual(block, residual, pre_weight, post_weight=None, gate=None, residual_scale=1.0, kind="rms",
                       pre_bias=None, post_bias=None, eps=1e-6):
    t = block if post_weight is None else norm(block, post_weight, post_bias, kind, eps)
    if gate is not None:
        g = gate.reshape(-1, gate.shape[-1])
        t = t * np.repeat(g, t.shape[0] // g.shape[0], axis=0)
    r = residual_scale * residual + t
    return r, norm(r, pre_weight, pre_bias, kind, eps)


def quantize_rows(x):
    """(codes as float64, scales float64); 16-bit inputs: the quotient's ties are exact in 64 bits."""
    top = np.abs(x).max(-1)
    safe = np.where(top == 0, 1.0, top)
    return np.rint(x * 127.0 / safe[:, None]), top / 127.0


def gemm_w8a8(q, q_scales, weight, weight_scales, bias=None):
    acc = q.astype(np.float64) @ weight.astype(np.float64).T       # integers below 2^31: exact
    y = acc * q_scales[:, None] * weight_scales[None, :]
    return y if bias is None else y + bias


# Half a unit in the last place, relative: what one rounding to the type may cost.
UNIT = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


def unit(dtype):
    return UNIT[str(dtype).replace("torch.", "")]


def route(logits, top_k, renormalize):
    """(ids [M][top_k], weights) in 64 bits, ties to the lowest index."""
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    e = np.exp(logits - logits.max(1, keepdims=True))
    chosen = np.take_along_axis(e, ids, 1)
    return ids, chosen / (chosen if renormalize else e).sum(1, keepdims=True)


def moe(x, router, gate, up, down, top_k, renormalize=True, inv_s=None):
    """gate, up, down: lists of dequantized float64 layers."""
    ids, p = route(x @ router.T, top_k, renormalize)
    xs = x if inv_s is None else x * inv_s
    y = np.zeros_like(x)
    for m in range(x.shape[0]):
        for e, w in zip(ids[m], p[m]):
            g, u = gate[e] @ xs[m], up[e] @ xs[m]
            y[m] += w * (down[e] @ (g / (1 + np.exp(-g)) * u))
    return y
