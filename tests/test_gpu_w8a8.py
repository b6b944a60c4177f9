"""GPU parity of awq_gemm_w8a8 and awq_linear_w8a8 against 64-bit forms.

The integer sum is exact, three fp32 roundings follow (two scales, the bias) and
one to the output's type: |y - ref| <= (u + 2^-22) |ref| + 2^-23 |bias| + tiny.
linear_w8a8 quantizes 16-bit rows, whose codes are the exact quotient's, so the
same bound holds for it.
"""
import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq

import block_reference as R
from gpu_util import announce, guarded_empty, sentinel_intact

pytestmark = pytest.mark.gpu


def dtype_of(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16}[name]


def codes(M, K, seed):
    import torch
    g = np.random.default_rng(seed)
    a = np.clip(np.rint(40 * g.standard_normal((M, K))), -127, 127).astype(np.int8)
    return torch.from_numpy(a).cuda()


def scales(M, seed, size):
    import torch
    g = np.random.default_rng(seed)
    return torch.from_numpy((size * np.exp(0.3 * g.standard_normal(M))).astype(np.float32)).cuda()


def check(y, ref, bias):
    extra = 0.0 if bias is None else 2.0 ** -23 * np.abs(R.to_f64(bias))[None, :]
    bound = (R.unit(y.dtype) + 2.0 ** -22) * np.abs(ref) + extra + 2.0 ** -24
    worst = np.max(np.abs(R.to_f64(y) - ref) / bound)
    assert worst <= 1.0, f"{worst:.3f} of the bound"


# (M, N, K).  One row to 64 (1, 2 and 4 row tiles), ragged rows, columns and last K steps (K % 128 of 16, 64,
# 112), one column, K cut into splits (few columns, long rows), full and ragged output tiles of the many-row
# kernels, M and N one past a tile
SHAPES = [(1, 1, 16), (1, 64, 128), (1, 4096, 4096), (1, 37, 28672), (2, 1000, 4096), (3, 130, 4112),
          (4, 300, 8192), (5, 96, 240), (13, 50, 2048), (16, 600, 1408), (17, 70, 11008), (31, 515, 4096),
          (33, 1030, 2160), (64, 256, 4096), (64, 48, 28672), (65, 300, 512), (127, 1000, 1024),
          (130, 257, 4096), (256, 256, 128), (257, 515, 1040), (509, 1024, 4096), (1000, 4100, 640),
          (2048, 2048, 512), (4100, 300, 8192),
          # workgroups of 8 waves for every compute unit at 5 to 64 rows, and codes that are split to fit in LDS
          (5, 24577, 144), (16, 24600, 256), (33, 24577, 272), (64, 24640, 528), (3, 4200, 28672), (4, 4096, 20496),
          (2, 2050, 65552), (1, 4099, 65568)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_w8a8(gpu, M, N, K, dtype):
    import torch
    announce("gemm_w8a8", f"M={M} N={N} K={K} {dtype} workspace={awq.gemm_w8a8_workspace_bytes(M, N, K)}")
    x, w = codes(M, K, 1), codes(N, K, 2)
    sx, sw = scales(M, 3, 0.02), scales(N, 4, 0.01 / np.sqrt(K))
    for bias in (None, scales(N, 5, 1.0)):
        y, raw, n = guarded_empty((M, N), dtype_of(dtype))
        awq.gemm_w8a8(x, sx, w, sw, bias=bias, out=y)
        torch.cuda.synchronize()
        assert sentinel_intact(raw, n)
        check(y, R.gemm_w8a8(x.cpu().numpy(), R.to_f64(sx), w.cpu().numpy(), R.to_f64(sw),
                             None if bias is None else R.to_f64(bias)), bias)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_w8a8(gpu, M, N, K, dtype):
    import torch
    announce("linear_w8a8", f"M={M} N={N} K={K} {dtype} workspace={awq.linear_w8a8_workspace_bytes(M, N, K)}")
    g = np.random.default_rng(M + N + K)
    x = torch.from_numpy((g.standard_normal((M, K)) * np.exp(0.5 * g.standard_normal(K))).astype(np.float32))
    x = x.to(dtype_of(dtype)).cuda()
    w, sw, bias = codes(N, K, 2), scales(N, 4, 0.01 / np.sqrt(K)), scales(N, 5, 1.0)
    y = awq.linear_w8a8(x, w, sw, bias=bias)
    q, s = awq.quantize_rows(x)
    y2 = awq.gemm_w8a8(q, s, w, sw, bias=bias, dtype=x.dtype)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
    qr, sr = R.quantize_rows(R.to_f64(x))
    check(y, R.gemm_w8a8(qr, sr, w.cpu().numpy(), R.to_f64(sw), R.to_f64(bias)), bias)


# (M, N, K) that take the 256 x 256 tiles: one, three and four K steps, ragged last steps and edges, more tiles than
# compute units (workgroups that take a second one), widths of 8-, 4- and 1-element alignment
WIDE = [(4352, 4352, 128), (4097, 4360, 384), (4400, 4701, 272), (300, 30004, 1040), (2049, 16392, 16),
        (8192, 4096, 528)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K", WIDE)
def test_gemm_w8a8_wide(gpu, M, N, K, dtype):
    import torch
    announce("gemm_w8a8 wide", f"M={M} N={N} K={K} {dtype}")
    x, w = codes(M, K, 1), codes(N, K, 2)
    sx, sw, bias = scales(M, 3, 0.02), scales(N, 4, 0.01 / np.sqrt(K)), scales(N, 5, 1.0)
    y, raw, n = guarded_empty((M, N), dtype_of(dtype))
    awq.gemm_w8a8(x, sx, w, sw, bias=bias, out=y)
    again = awq.gemm_w8a8(x, sx, w, sw, bias=bias, dtype=dtype_of(dtype))
    torch.cuda.synchronize()
    assert sentinel_intact(raw, n)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    # integers below 2^31 in 64 bits on the GPU: the reference of every output, without 4 GB of host arrays
    acc = torch.round(x.double() @ w.double().t())
    ref = acc * sx.double()[:, None] * sw.double()[None, :] + bias.double()[None, :]
    bound = (R.unit(y.dtype) + 2.0 ** -22) * ref.abs() + 2.0 ** -23 * bias.double().abs()[None, :] + 2.0 ** -24
    worst = ((y.double() - ref).abs() / bound).max().item()
    assert worst <= 1.0, f"{worst:.3f} of the bound"


@pytest.mark.parametrize("M,N", [(1, 64), (12, 64), (64, 64), (300, 512)])
def test_largest_sums_are_exact(gpu, M, N):
    """Codes at the ends of their range over the longest K: the sum stays below 2^31."""
    import torch
    K = (1 << 17) - 16
    x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one_m, one_n = torch.full((M,), 2.0 ** -20, device="cuda"), torch.ones(N, device="cuda")
    y = awq.gemm_w8a8(x, one_m, w, one_n)
    ref = np.where(np.arange(N) % 2 == 0, 128.0 * 128 * K, -128.0 * 127 * K) * 2.0 ** -20
    check(y, np.broadcast_to(ref, (M, N)), None)


def test_zero_scale_and_bad_rows(gpu):
    """A row of zeros gives the bias; a NaN row stays in its row."""
    import torch
    for M in (4, 200):
        x = torch.randn(M, 512, device="cuda").half()
        x[0] = 0
        w, sw, bias = codes(96, 512, 2), scales(96, 3, 0.01), scales(96, 4, 1.0)
        y0 = awq.linear_w8a8(x, w, sw, bias=bias)
        x[2, 7] = float("nan")
        y = awq.linear_w8a8(x, w, sw, bias=bias)
        assert torch.equal(y[0], bias.half())
        keep = [m for m in range(M) if m != 2]
        assert torch.equal(y[keep], y0[keep]) and torch.isnan(y[2]).all()


def test_weights_past_32_bit_offsets(gpu):
    """A weight matrix of more than 2^31 bytes: the last columns are the right ones."""
    import torch
    K, N = 65536, 33000
    w = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    w[-5:] = codes(5, K, 1)
    sw = torch.full((N,), 1e-4, device="cuda")
    for M in (1, 70):
        x, sx = codes(M, K, 2), scales(M, 3, 0.01)
        y = awq.gemm_w8a8(x, sx, w, sw)
        assert not y[:, :-5].any()
        check(y[:, -5:], R.gemm_w8a8(x.cpu().numpy(), R.to_f64(sx), w[-5:].cpu().numpy(), np.full(5, np.float32(1e-4))),
              None)


def test_own_workspace_and_stream(gpu):
    """A caller's workspace on another stream, and the same bits again."""
    import torch
    M, N, K = 16, 64, 28672
    x, w, sx, sw = codes(M, K, 1), codes(N, K, 2), scales(M, 3, 0.02), scales(N, 4, 1e-4)
    need = awq.gemm_w8a8_workspace_bytes(M, N, K)
    assert need > 0
    y0 = awq.gemm_w8a8(x, sx, w, sw)
    torch.cuda.synchronize()
    ws = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        y = awq.gemm_w8a8(x, sx, w, sw, workspace=ws)
    st.synchronize()
    assert torch.equal(y, y0)
    with pytest.raises(awq.AwqError):
        awq.gemm_w8a8(x, sx, w, sw, workspace=ws[: need // 2])


def test_refusals(gpu):
    import torch
    x, w, sx, sw = codes(4, 512, 1), codes(64, 512, 2), scales(4, 3, 1.0), scales(64, 4, 1.0)
    with pytest.raises(TypeError):
        awq.gemm_w8a8(x.half(), sx, w, sw)
    with pytest.raises(TypeError):
        awq.gemm_w8a8(x, sx.half(), w, sw)
    with pytest.raises(TypeError):
        awq.gemm_w8a8(x, sx, w, sw, dtype=torch.float32)
    with pytest.raises(ValueError):
        awq.gemm_w8a8(x, sx, w[:, :496], sw)
    with pytest.raises(ValueError):
        awq.gemm_w8a8(x, sx, w, sw[:63])
    with pytest.raises(ValueError):
        awq.gemm_w8a8(x, sx, w.t().contiguous().t(), sw)
    with pytest.raises(ValueError):
        awq.linear_w8a8(x.half(), w, sw, bias=sw.cpu())
    with pytest.raises(awq.AwqError):
        awq.gemm_w8a8(codes(4, 520, 1), sx, codes(64, 520, 1), sw)
    e = torch.empty(0, 512, dtype=torch.int8, device="cuda")
    assert awq.gemm_w8a8(e, sx[:0], w, sw).shape == (0, 64)
    assert awq.linear_w8a8(x.half(), w[:0], sw[:0]).shape == (4, 0)
