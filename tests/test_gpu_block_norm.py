"""GPU parity of awq_norm_gate_residual and awq_quantize_rows against 64-bit
forms.

Bounds, per element.  r' = alpha r + g t and h are computed in fp32 and rounded
once: |out - ref| <= u |ref| + c with u half a unit of the type and c the fp32
error.  A mean over H <= 32768 values is off by at most (H / threads + 20)
2^-24 of the mean magnitude, and the norms multiply a handful of fp32 terms:
c = 2^-16 of the row's largest |ref| covers both for every H here (a row's
values may cancel in alpha r + g t, so c goes by the row, not by the element).
Codes equal the 64-bit ones exactly for 16-bit rows; behind a norm the fp32 h
may sit on the other side of a half-integer, so there a code may differ by one
where the 64-bit quotient is within 127 * 2^-16 of half way.
"""
import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq

import block_reference as R
from gpu_util import announce, guarded_empty, sentinel_intact

pytestmark = pytest.mark.gpu
FP32 = 2.0 ** -16


def torch_dtype(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16}[name]


def rows(T, H, seed, dtype, scale=1.0):
    import torch
    g = np.random.default_rng(seed)
    a = g.standard_normal((T, H)) * np.exp(0.5 * g.standard_normal(H)) * scale
    return torch.from_numpy(a.astype(np.float32)).to(torch_dtype(dtype)).cuda()


def vector(H, seed, dtype, mean=1.0, std=0.2, n=None):
    import torch
    g = np.random.default_rng(seed)
    a = mean + std * g.standard_normal((n, H) if n else H)
    return torch.from_numpy(a.astype(np.float32)).to(torch_dtype(dtype)).cuda()


def f64(t):
    return None if t is None else R.to_f64(t)


def check(out, ref, dtype, what):
    got = R.to_f64(out)
    bound = R.unit(out.dtype) * np.abs(ref) + FP32 * np.abs(ref).max(-1, keepdims=True) + 2.0 ** -24
    worst = np.max(np.abs(got - ref) / bound)
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


# (T, H): one chunk, part of a wave, one and two chunks per lane, every workgroup size on either side of its
# border, odd row counts, the widest row, more rows than compute units
SHAPES = [(1, 8), (3, 256), (1, 520), (5, 1024), (2, 2048), (7, 2056), (1, 4096), (300, 4096), (2, 8192),
          (259, 8192), (3, 8200), (1, 16392), (2, 32768)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_gate_residual(gpu, T, H, kind, dtype):
    import torch
    announce("norm_gate_residual", f"T={T} H={H} {kind} {dtype}")
    block, residual = rows(T, H, 1, dtype), rows(T, H, 2, dtype, 4.0)
    pre, post = vector(H, 3, dtype), vector(H, 4, dtype, 0.5, 0.1)
    prb, pob = vector(H, 5, dtype, 0.0, 0.1), vector(H, 6, dtype, 0.0, 0.1)
    gates = [None, vector(H, 7, dtype, 0.0, 0.7), vector(H, 8, dtype, 0.0, 0.7, n=T)]
    options = [dict(), dict(post_weight=post), dict(post_weight=post, post_bias=pob, pre_bias=prb)]
    for i, opt in enumerate(options):
        for gate, alpha in zip(gates, (1.0, 0.7, -1.25)):
            raw = [guarded_empty((T, H), block.dtype) for _ in range(2)]
            r, h = awq.norm_gate_residual(block, residual, pre, gate=gate, residual_scale=alpha, kind=kind,
                                          eps=1e-5, out=(raw[0][0], raw[1][0]), **opt)
            torch.cuda.synchronize()
            assert all(sentinel_intact(x, n) for _, x, n in raw)
            rr, hr = R.norm_gate_residual(f64(block), f64(residual), f64(pre), gate=f64(gate),
                                          residual_scale=np.float32(alpha), kind=kind, eps=1e-5,
                                          **{k: f64(v) for k, v in opt.items()})
            check(r, rr, dtype, f"r' {i}")
            check(h, hr, dtype, f"h {i}")


def test_gate_rows_cover_consecutive_rows(gpu):
    block, residual = rows(12, 512, 1, "fp16"), rows(12, 512, 2, "fp16")
    gate, pre = vector(512, 3, "fp16", n=4), vector(512, 4, "fp16")
    r, _ = awq.norm_gate_residual(block, residual, pre, gate=gate)
    check(r, R.norm_gate_residual(f64(block), f64(residual), f64(pre), gate=f64(gate))[0], "fp16", "r'")


def test_in_place_residual_and_repeat(gpu):
    """`residual` may be the output, and the same call gives the same bits."""
    import torch
    block, residual, pre = rows(9, 4096, 1, "bf16"), rows(9, 4096, 2, "bf16"), vector(4096, 3, "bf16")
    r0, h0 = awq.norm_gate_residual(block, residual, pre)
    h = torch.empty_like(block)
    r, h = awq.norm_gate_residual(block, residual, pre, out=(residual, h))
    assert r is residual
    assert torch.equal(r.view(torch.int16), r0.view(torch.int16))
    assert torch.equal(h.view(torch.int16), h0.view(torch.int16))


def test_a_large_mean_does_not_cancel(gpu):
    """Layer norm of rows whose mean is 500 times their spread."""
    import torch
    g = np.random.default_rng(0)
    block = torch.zeros(4, 4096, dtype=torch.bfloat16, device="cuda")
    residual = torch.from_numpy((500 + g.standard_normal((4, 4096))).astype(np.float32)).to(torch.float16).cuda()
    pre = vector(4096, 3, "fp16")
    _, h = awq.norm_gate_residual(block.half(), residual, pre, kind="layer")
    check(h, R.norm_gate_residual(np.zeros((4, 4096)), f64(residual), f64(pre), kind="layer")[1], "fp16", "h")


def test_zero_rows(gpu):
    """A row of zeros: eps keeps the norm finite, its codes and scale are zero."""
    import torch
    z = torch.zeros(2, 1024, dtype=torch.float16, device="cuda")
    one = torch.ones(1024, dtype=torch.float16, device="cuda")
    r, h = awq.norm_gate_residual(z, z, one, post_weight=one)
    assert not r.any() and not h.any()
    r, q, s = awq.norm_gate_residual(z, z, one, quantize=True)
    assert not q.any() and not s.any()


def test_bad_rows_stay_in_their_row(gpu):
    """An infinity or a NaN spoils its own row and no other."""
    import torch
    block, residual, pre = rows(6, 2048, 1, "fp16"), rows(6, 2048, 2, "fp16"), vector(2048, 3, "fp16")
    r0, h0 = awq.norm_gate_residual(block, residual, pre)
    block[1, 5] = float("inf")
    block[4, 2047] = float("nan")
    r, h = awq.norm_gate_residual(block, residual, pre)
    keep = [0, 2, 3, 5]
    assert torch.equal(h[keep], h0[keep]) and torch.equal(r[keep], r0[keep])
    assert torch.isinf(r[1, 5]) and torch.isnan(h[1, 5]) and torch.isnan(h[4]).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,H", [(1, 64), (3, 1040), (5, 4096), (300, 8192), (2, 16400)])
def test_norm_with_codes(gpu, T, H, dtype):
    import torch
    announce("norm codes", f"T={T} H={H} {dtype}")
    block, residual, pre = rows(T, H, 1, dtype), rows(T, H, 2, dtype, 4.0), vector(H, 3, dtype)
    r, q, s = awq.norm_gate_residual(block, residual, pre, quantize=True)
    r0, h0 = awq.norm_gate_residual(block, residual, pre)
    assert torch.equal(r.view(torch.int16), r0.view(torch.int16))
    href = R.norm_gate_residual(f64(block), f64(residual), f64(pre))[1]
    qr, sr = R.quantize_rows(href)
    assert np.all(np.abs(R.to_f64(s) - sr) <= 2.0 ** -16 * sr)
    off = R.to_f64(q) - qr
    t = href * 127.0 / np.abs(href).max(-1, keepdims=True)
    near = np.abs(np.abs(t - np.floor(t)) - 0.5) <= 127 * FP32
    assert np.all((off == 0) | (near & (np.abs(off) == 1)))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 16), (5, 512), (3, 1040), (2, 4096), (300, 4096), (2, 28672), (1, 32784),
                                 (3, 65536)])
def test_quantize_rows(gpu, M, K, dtype):
    """Codes of the exact quotient, ties to even, and the rounded scale."""
    import torch
    announce("quantize_rows", f"M={M} K={K} {dtype}")
    x = rows(M, K, M + K, dtype)
    x[0, : K // 2] = torch.round(x[0, : K // 2] * 2) / 2          # many ties
    x[0, 0] = 127.0
    raw_q, raw_s = guarded_empty((M, K), torch.int8), guarded_empty((M,), torch.float32)
    q, s = awq.quantize_rows(x, out=(raw_q[0], raw_s[0]))
    torch.cuda.synchronize()
    assert sentinel_intact(*raw_q[1:]) and sentinel_intact(*raw_s[1:])
    qr, sr = R.quantize_rows(f64(x))
    assert np.array_equal(R.to_f64(q), qr)
    assert np.array_equal(s.cpu().numpy(), (np.abs(f64(x)).max(-1).astype(np.float32) / np.float32(127)))


def test_quantize_rows_extremes(gpu):
    """Zeros, the smallest and largest magnitudes, an infinity and a NaN."""
    import torch
    x = torch.zeros(6, 64, dtype=torch.bfloat16, device="cuda")
    x[1, 3] = 1e-40
    x[1, 4] = -5e-41
    x[2] = 3.0e38
    x[2, 0] = -3.0e38
    x[3, 7] = float("inf")
    x[4, 9] = float("nan")
    x[5] = -1.0
    q, s = awq.quantize_rows(x)
    assert not q[0].any() and s[0] == 0
    # bfloat16 holds both as the same subnormal: the codes are those of the stored values
    assert np.array_equal(R.to_f64(q[1:2]), R.quantize_rows(f64(x[1:2]))[0]) and q[1, 3] == 127 and s[1] > 0
    assert q[2, 0] == -127 and (q[2, 1:] == 127).all() and torch.isfinite(s[2])
    assert torch.isinf(s[3]) and torch.isnan(s[4])
    assert (q[5] == -127).all()


# Rows of 64 around a maximum of 2^e (nearly 2^(e + 1) in "full"): half of it (a quotient of 63.5), quarters, tenths
# and halves of every size down to 2^-32 of it, and the smallest numbers
LARGE = [118, 119, 120, 121, 122, 125, 126, 127]


def large_rows():
    import torch
    g = np.random.default_rng(0)
    out = []
    for e in LARGE:
        for top in (1.0, 2.0 - 2.0 ** -7):
            row = np.concatenate([[1, .5, .25, -.75, .1, -1, 0, .3], 2.0 ** -np.arange(1, 33), [1e-30, -1e-30],
                                  (np.arange(14) - 7 + 0.5) / 127, g.uniform(-1, 1, 8)])
            out.append(row * top * 2.0 ** e)
    x = torch.tensor(np.stack(out), dtype=torch.float64).to(torch.bfloat16)
    x[:, 62] = 2.0 ** -130
    x[:, 63] = -2.0 ** -133
    return x.cuda()


def test_codes_of_large_rows(gpu):
    """bfloat16 rows up to the largest finite numbers: 127 v is past fp32 there, the quotient is not."""
    x = large_rows()
    qr, sr = R.quantize_rows(f64(x))
    q, s = awq.quantize_rows(x)
    assert np.array_equal(R.to_f64(q), qr)
    assert np.array_equal(s.cpu().numpy(), np.abs(f64(x)).max(-1).astype(np.float32) / np.float32(127))


@pytest.mark.parametrize("M", [1, 2])
def test_large_rows_quantized_inside_the_product(gpu, M):
    """The same codes where the product's own launch quantizes one or two rows: an identity for weights, whose
    channel scales bring the outputs to the codes times fp32 factors (three roundings of 2^-24 and bfloat16's)."""
    import torch
    x = large_rows()
    w, sw = torch.eye(64, dtype=torch.int8, device="cuda"), torch.full((64,), 2.0 ** -100, device="cuda")
    assert awq.linear_w8a8_workspace_bytes(M, 64, 64) == 0
    qr, sr = R.quantize_rows(f64(x))
    for m in range(0, len(x), M):
        y = awq.linear_w8a8(x[m:m + M], w, sw)
        ref = qr[m:m + M] * sr[m:m + M, None] * 2.0 ** -100
        assert np.all(np.abs(R.to_f64(y) - ref) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(ref))


def test_norm_codes_of_large_rows(gpu):
    """The same behind a norm whose weights are as large: a row of ones of either sign, so h is +-weight within
    2^-16 and a code may differ by one where the quotient is that near half way."""
    import torch
    w = large_rows()
    signs = torch.where(torch.arange(64, device="cuda") % 3 == 0, -1.0, 1.0).to(torch.bfloat16)[None]
    for k in range(len(w)):
        r, q, s = awq.norm_gate_residual(torch.zeros_like(signs), signs, w[k], eps=0.0, quantize=True)
        href = R.norm_gate_residual(np.zeros((1, 64)), f64(signs), f64(w[k]), eps=0.0)[1]
        qr, sr = R.quantize_rows(href)
        t = href * 127.0 / np.abs(href).max()
        near = np.abs(np.abs(t - np.floor(t)) - 0.5) <= 127 * FP32
        off = R.to_f64(q) - qr
        assert np.all((off == 0) | (near & (np.abs(off) == 1)))
        assert np.all(np.abs(R.to_f64(s) - sr) <= FP32 * sr)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,H", [(300, 16384), (257, 24576), (40, 512), (300, 1536)])
def test_widths_in_more_rows_than_compute_units(gpu, T, H, dtype):
    """The widest rows where there are many of them, in 16 bits and as codes, and the narrow ones."""
    block, residual, pre = rows(T, H, 1, dtype), rows(T, H, 2, dtype, 4.0), vector(H, 3, dtype)
    r, h = awq.norm_gate_residual(block, residual, pre, kind="layer")
    rr, hr = R.norm_gate_residual(f64(block), f64(residual), f64(pre), kind="layer")
    check(r, rr, dtype, "r'")
    check(h, hr, dtype, "h")
    q, s = awq.quantize_rows(block)
    qr, sr = R.quantize_rows(f64(block))
    assert np.array_equal(R.to_f64(q), qr)
    assert np.array_equal(s.cpu().numpy(), np.abs(f64(block)).max(-1).astype(np.float32) / np.float32(127))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,H", [(1, 520), (6, 4096), (300, 2048), (260, 8192)])
def test_every_norm_with_codes(gpu, T, H, kind, dtype):
    """Codes behind norms with a norm after the block, gates and biases.  h and the row's maximum are both off by at
    most 2^-16 of that maximum: a quotient by 2 * 127 * 2^-16."""
    import torch
    block, residual = rows(T, H, 1, dtype), rows(T, H, 2, dtype, 4.0)
    pre, post = vector(H, 3, dtype), vector(H, 4, dtype, 0.5, 0.1)
    opt = dict(post_weight=post, gate=vector(H, 7, dtype, 0.0, 0.7), pre_bias=vector(H, 5, dtype, 0.0, 0.1),
               post_bias=vector(H, 6, dtype, 0.0, 0.1))
    r, q, s = awq.norm_gate_residual(block, residual, pre, kind=kind, residual_scale=0.7, quantize=True, **opt)
    r0, _ = awq.norm_gate_residual(block, residual, pre, kind=kind, residual_scale=0.7, **opt)
    assert torch.equal(r.view(torch.int16), r0.view(torch.int16))
    href = R.norm_gate_residual(f64(block), f64(residual), f64(pre), kind=kind, residual_scale=np.float32(0.7),
                                **{k: f64(v) for k, v in opt.items()})[1]
    qr, sr = R.quantize_rows(href)
    assert np.all(np.abs(R.to_f64(s) - sr) <= FP32 * sr + 2.0 ** -23 * sr)
    off = R.to_f64(q) - qr
    t = href * 127.0 / np.abs(href).max(-1, keepdims=True)
    near = np.abs(np.abs(t - np.floor(t)) - 0.5) <= 2 * 127 * FP32
    assert np.all((off == 0) | (near & (np.abs(off) == 1)))


def test_more_rows_than_a_launch_holds(gpu):
    """2^26 rows and a few: 2^32 threads of the narrowest workgroups.  Every row has codes of its own."""
    import torch
    M = (1 << 26) + 3
    announce("quantize_rows", f"M={M} K=16")
    x = torch.zeros(M, 16, dtype=torch.float16, device="cuda")
    t = torch.arange(M, device="cuda")
    x[:, 5] = (t % 251 - 125).half()
    x[:, 15] = 127.0
    q, s = awq.quantize_rows(x)
    assert bool((s == 1.0).all()) and bool((q[:, 15] == 127).all()) and bool((q[:, 5] == (t % 251 - 125)).all())
    assert not q[:, :5].any() and not q[:, 6:15].any()
    del x, q, s
    announce("norm_gate_residual", f"T={M} H=8")
    residual = torch.zeros(M, 8, dtype=torch.float16, device="cuda")
    residual[:, 0] = (t % 2048 + 1).half()
    gate = torch.tensor([[1.0], [2.0], [3.0]], device="cuda").repeat_interleave(8, dim=1).half().contiguous()
    n = M // 3 * 3                                           # three gate rows
    r, h = awq.norm_gate_residual(torch.ones_like(residual)[:n], residual[:n], torch.ones(8, device="cuda").half(),
                                  gate=gate, eps=0.0)
    g = torch.arange(n, device="cuda") // (n // 3) + 1
    assert bool((r[:, 1] == g.half()).all()) and bool((r[:, 0] == (t[:n] % 2048 + 1 + g).half()).all())
    # h = r' / sqrt((r0^2 + 7 g^2) / 8), one rounding of fp16 (2^-11) past fp32's
    ref = g.float() * torch.rsqrt(((t[:n] % 2048 + 1 + g).float() ** 2 + 7 * g.float() ** 2) / 8)
    assert bool(((h[:, 7].float() - ref).abs() <= ref * 2.0 ** -10 + 2.0 ** -24).all())


def test_refusals(gpu):
    import torch
    b, w = rows(4, 512, 1, "fp16"), vector(512, 2, "fp16")
    with pytest.raises(TypeError):
        awq.norm_gate_residual(b.float(), b, w)
    with pytest.raises(TypeError):
        awq.norm_gate_residual(b, b.bfloat16(), w)
    with pytest.raises(ValueError):
        awq.norm_gate_residual(b[0], b, w)
    with pytest.raises(ValueError):
        awq.norm_gate_residual(b, b[:3], w)
    with pytest.raises(ValueError):
        awq.norm_gate_residual(b[:, ::2], b[:, ::2], w[::2])
    with pytest.raises(ValueError):
        awq.norm_gate_residual(b, b, w, post_bias=w)
    with pytest.raises(ValueError):
        awq.norm_gate_residual(b, b, w, kind="batch")
    with pytest.raises(ValueError):
        awq.norm_gate_residual(b, b, w, gate=vector(512, 3, "fp16", n=3))
    with pytest.raises(ValueError):
        awq.norm_gate_residual(b.cpu(), b, w)
    with pytest.raises(awq.AwqError):
        awq.norm_gate_residual(b[:, :508].contiguous(), b[:, :508].contiguous(), w[:508].contiguous())
    with pytest.raises(awq.AwqError):
        awq.norm_gate_residual(b, b, w, eps=-1.0)
    with pytest.raises(awq.AwqError):
        awq.quantize_rows(b[:, :504].contiguous())
    with pytest.raises(TypeError):
        awq.quantize_rows(b.float())
    e = torch.empty(0, 512, dtype=torch.float16, device="cuda")
    r, h = awq.norm_gate_residual(e, e, w)
    assert r.shape == h.shape == (0, 512)
    q, s = awq.quantize_rows(e)
    assert q.shape == (0, 512) and s.shape == (0,)


def test_mean_squares_past_fp32(gpu):
    """bfloat16 rows whose squares overflow are divided by infinity: the bias is what is left, and no other row
    changes."""
    import torch
    block, residual, pre = rows(3, 512, 1, "bf16"), rows(3, 512, 2, "bf16"), vector(512, 3, "bf16")
    bias = vector(512, 4, "bf16", 0.0, 0.5)
    _, h0 = awq.norm_gate_residual(block, residual, pre, pre_bias=bias)
    residual[1] = 1e20
    _, h = awq.norm_gate_residual(block, residual, pre, pre_bias=bias)
    assert torch.equal(h[1], bias) and torch.equal(h[[0, 2]], h0[[0, 2]])
