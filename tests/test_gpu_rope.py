"""GPU parity of awq_rope against 64 bits.

Angles are 64-bit products, so the sine and cosine are fp32's of the right angle: within 2^-22 with the
rounding of the fraction of a turn (2^-24 of a turn, 2 pi 2^-25 radians), its sine (2^-23) and the magnitude's
product.  A pair's turn adds two fp32 roundings, then one to the type:
|y - ref| <= u |ref| + 2^-20.5 m (|a| + |b|) + tiny.
"""
import numpy as np
import pytest

import weight_only_quantization_pack_amd as awq

import block_reference as R
import cache_reference as C
from cache_util import DTYPES, dtype_of, freq, gpu as put, ints
from gpu_util import announce, guarded_empty, sentinel_intact

pytestmark = pytest.mark.gpu


def rows(T, heads, dim, dtype, seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((T, heads, dim)) * np.exp(0.5 * g.standard_normal((heads, dim)))
    return put(x.astype(np.float32)).to(dtype_of(dtype))


def check(y, x, positions, inv_freq, magnitude, layout, inverse=False):
    xs, f = R.to_f64(x), inv_freq.cpu().numpy()
    ref = C.rope(xs, positions, f, magnitude, layout, inverse)
    n = len(f)
    a, b = (np.s_[..., :n], np.s_[..., n:2 * n]) if layout == "half" else (np.s_[..., 0:2 * n:2], np.s_[..., 1:2 * n:2])
    pair = np.zeros_like(xs)
    pair[a] = pair[b] = np.abs(xs[a]) + np.abs(xs[b])
    bound = R.unit(y.dtype) * np.abs(ref) + 2.0 ** -20.5 * magnitude * pair + 2.0 ** -24
    worst = np.max(np.abs(R.to_f64(y) - ref) / bound)
    assert worst <= 1.0, f"{worst:.3f} of the bound"
    assert np.array_equal(R.to_f64(y)[..., 2 * n:], xs[..., 2 * n:])      # what is not turned is copied


SHAPES = [(1, 1, 16, 16), (1, 32, 128, 128), (2, 3, 64, 32), (5, 7, 96, 48), (3, 2, 80, 16), (4, 5, 256, 256),
          (7, 1, 512, 512), (9, 40, 128, 64), (130, 8, 192, 192), (1027, 6, 64, 64)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,heads,dim,rotary", SHAPES)
def test_rope(gpu, T, heads, dim, rotary, dtype, layout):
    import torch
    announce("rope", T, heads, dim, rotary, dtype, layout)
    x = rows(T, heads, dim, dtype, T + heads + dim)
    positions = np.random.default_rng(T).integers(0, 1 << 17, T).astype(np.int32)
    f, m = freq(rotary)
    out, raw, n = guarded_empty((T, heads, dim), x.dtype)
    awq.rope(x, put(positions), f, layout=layout, out=out)
    torch.cuda.synchronize()
    assert sentinel_intact(raw, n)
    check(out, x, positions, f, m, layout)


@pytest.mark.parametrize("positions", [[0, 1, -1, 2, -7], [1 << 20, (1 << 20) + 1, 999983, 123456789, (1 << 31) - 1],
                                       [-(1 << 31), 5, 5, 5, 0]])
def test_far_and_negative_positions(gpu, positions):
    """Exact in 64 bits but for their product: 2^31 * f is held to 2^-21 of a turn at worst, which the bound has
    no room for, so these frequencies end in few bits."""
    announce("rope positions", positions)
    x = rows(5, 4, 64, "fp16", 1)
    f = put((2.0 ** -np.arange(32) * 1.25).astype(np.float32))
    p = np.array(positions, dtype=np.int64).astype(np.int32)
    check(awq.rope(x, put(p), f), x, p, f, 1.0, "half")


def test_scaled_strided_in_place_and_back(gpu):
    import torch
    announce("rope scaled, strided, in place, inverse")
    f, m = freq(64, 500000.0, scaling="yarn", factor=16.0, original_length=4096.0)
    qkv = rows(33, 12, 64, "bf16", 2)                       # [q | k | v] of one projection
    keep = qkv.clone()
    p = np.arange(33, dtype=np.int32) + 70000
    q, k = qkv[:, :8], qkv[:, 8:10]
    got = awq.rope(k, put(p), f, layout="interleaved", magnitude=m)
    check(got, k, p, f, m, "interleaved")
    awq.rope(q, put(p), f, magnitude=m, out=q)
    check(q, keep[:, :8], p, f, m, "half")
    assert torch.equal(qkv[:, 8:], keep[:, 8:])             # the neighbours are left alone
    x = keep[:, :8].contiguous().half()
    turned = awq.rope(x, put(p), f, magnitude=m)
    back = awq.rope(turned, put(p), f, magnitude=m, inverse=True)
    check(back, turned, p, f, m, "half", inverse=True)
    # turning back undoes the turn, times the magnitude twice
    assert float((back.double() / m ** 2 - x.double()).abs().max() / x.double().abs().max()) < 4 * 2.0 ** -11


def test_inverse_is_the_gradient(gpu):
    """<rope(x), g> changes along dx by <dx, rope^-1(g)>: against differences in 64 bits."""
    f, _ = freq(48)
    x, g = rows(6, 3, 96, "bf16", 3), rows(6, 3, 96, "bf16", 4)
    p = np.array([0, 3, 17, 1000, 65535, 9], dtype=np.int32)
    got = R.to_f64(awq.rope(g, put(p), f, inverse=True))
    fs = f.cpu().numpy()
    base, e = R.to_f64(x), 1e-3
    r = np.random.default_rng(5)
    for _ in range(20):
        d = np.zeros_like(base)
        at = tuple(r.integers(0, n) for n in d.shape)
        d[at] = e
        diff = ((C.rope(base + d, p, fs) - C.rope(base - d, p, fs)) * R.to_f64(g)).sum() / (2 * e)
        assert abs(got[at] - diff) <= 2.0 ** -8 * abs(diff) + 1e-5 * np.abs(R.to_f64(g)).max()


def test_refused(gpu):
    import torch
    x = rows(4, 2, 64, "fp16", 6)
    f, _ = freq(64)
    p = ints([1, 2, 3, 4])
    for bad in (lambda: awq.rope(x.float(), p, f), lambda: awq.rope(x, p.long(), f), lambda: awq.rope(x, p, f.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: awq.rope(x[0], p, f), lambda: awq.rope(x, p[:3], f), lambda: awq.rope(x, p, f, layout="both"),
                lambda: awq.rope(x.transpose(1, 2), p, f), lambda: awq.rope(x, p, f, out=x[:3]),
                lambda: awq.rope(x, p.cpu(), f)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: awq.rope(x, p, freq(80)[0]), lambda: awq.rope(x, p, f[:4]),
                lambda: awq.rope(torch.zeros(4, 4, 66, dtype=torch.float16, device="cuda")[..., :64], p, f)):
        with pytest.raises((awq.AwqError, ValueError)):
            bad()
    assert awq.rope(x[:0], p[:0], f).shape == (0, 2, 64)
