"""Inputs, 64-bit references and error bounds for the products of two 8-bit
operands (not a test module).

Products of two e4m3 codes are exact, a scale block's products are summed in
f32 and the block's sum times both scales is added in f32: as in linear_util,
a sum of total magnitude m is off by at most (I + 16) 2^-24 m.

The e4m3 matrix instructions, which many rows of a bfloat16 product take, add a
rounding of their own: of eight consecutive columns' products each is cut to a
multiple of 2^(e - 13), e the largest exponent among them, a product's exponent
being the sum of its codes' (-6 for subnormal codes and zero).  So each loses less
than 2^-13 of (largest |x|, or 2^-6) times (largest |w|, or 2^-6) of the eight, in
codes; the largest itself keeps its 8 bits.  The codes of the tests' blocks reach 1
at least, so 2^-6 of a block's largest value stands for 2^-6 times its scale.
"""
import numpy as np
import torch

from linear_util import HALF, U, _act, assert_within, rel_l2  # noqa: F401

FINITE = np.array([c for c in range(256) if c & 127 != 127], np.uint8)


def weights(lead, O, I, seed):
    """codes u8 [*lead, O, I] of every finite value, scales over two decades."""
    r = np.random.default_rng(seed)
    w = FINITE[r.integers(0, 254, (*lead, O, I))]
    s = np.exp(r.uniform(np.log(1e-4), np.log(1e-2), (*lead, -(-O // 128), -(-I // 128))))
    return w, s.astype(np.float32)


def values(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()


def decode_weights(w, s):
    sc = np.repeat(np.repeat(s.astype(np.float64), 128, -2), 128, -1)
    return values(w) * sc[..., :w.shape[-2], :w.shape[-1]]


def decode_rows(codes, scales):
    """f64 torch [S][I] of quantized activations (numpy or torch)."""
    c = codes.cpu().numpy() if isinstance(codes, torch.Tensor) else codes
    s = scales.cpu().double().numpy() if isinstance(scales, torch.Tensor) else scales.astype(float)
    return torch.from_numpy(values(c) * np.repeat(s, 128, -1)[:, :c.shape[1]])


def rows(S, I, seed, outliers=True):
    """Quantized N(0,1) with a few outlier columns: codes u8, scales f32 (numpy)."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((S, I))
    if outliers:
        x *= np.where(r.random(I) < 0.01, 20.0, 1.0)
    return quantize(torch.from_numpy(x).float())


def quantize(x):
    """The definition: f32 scales, and the e4m3 values nearest to the exact quotients
    448 x / max|x|.  In 64 bits 448 x is exact, and the division's rounding cannot
    reach the middle of two codes, from which any other quotient of f32 numbers is
    2^-32 away at least; dividing by a power of two and rint are exact."""
    x = x.float()
    S, I = x.shape
    n = -(-I // 128)
    wide = torch.zeros(S, n * 128)
    wide[:, :I] = x
    b = wide.reshape(S, n, 128)
    m = b.abs().amax(2)
    s = (m / 448.0).clamp_min(2.0 ** -126)
    q = b.double() * 448.0 / m.double().clamp_min(448.0 * 2.0 ** -126)[:, :, None]
    step = torch.exp2(torch.frexp(q)[1].clamp_min(-5).double() - 4)
    q = torch.where(torch.isfinite(q), torch.round(q / step) * step, q)
    q = q.float().to(torch.float8_e4m3fn).view(torch.uint8)
    bad = ~torch.isfinite(b).all(2)             # an infinity or NaN in the block
    s[bad] = float("nan")
    q[bad] = 0x7F
    return q.reshape(S, -1)[:, :I].contiguous().numpy(), s.numpy()


def sum_bound(W, x, dtype):
    """How far the sums x W^T of a product with results of this type may be off
    (torch f64)."""
    W = torch.from_numpy(np.ascontiguousarray(W))
    bound = (W.shape[1] + 16) * U * (x.abs() @ W.abs().t())
    if dtype == torch.bfloat16:
        def largest(t):
            n = t.shape[0], -(-t.shape[1] // 128)
            wide = torch.zeros(n[0], n[1] * 128, dtype=t.dtype)
            wide[:, :t.shape[1]] = t.abs()
            block = wide.reshape(*n, 128).amax(2) * 2.0 ** -6
            return torch.maximum(wide.reshape(*n, 16, 8).amax(3), block[:, :, None]).flatten(1)
        bound = bound + 7 * 2.0 ** -13 * largest(x) @ largest(W).t()
    return bound


def reference(W, x, dtype, bias=None, act=None, gated=False, residual=None):
    """(y, bound) in f64 for decoded W [O][I] (numpy) and x [S][I] (torch f64)."""
    da = sum_bound(W, x, dtype)
    a = x @ torch.from_numpy(np.ascontiguousarray(W)).t()
    if bias is not None:
        a = a + bias.cpu().double()
        da = da + 2 * U * (a.abs() + bias.cpu().double().abs())
    v, dv = a, da
    if gated:
        h = a.shape[1] // 2
        up, dup = a[:, h:], da[:, h:]
        g = _act(a[:, :h], act)
        dg = 1.13 * da[:, :h] + 16 * U * (a[:, :h].abs() + g.abs())
        v = g * up
        dv = dg * (up.abs() + dup) + g.abs() * dup + U * v.abs()
    elif act is not None:
        v = _act(a, act)
        dv = 1.13 * da + 16 * U * (a.abs() + v.abs())
    if residual is not None:
        r = residual.cpu().double()
        v = v + r
        dv = dv + U * (v.abs() + dv)
    # an f32 below 2^-126 may be flushed
    return v, dv + HALF[dtype] * (v.abs() + dv) + 2.0 ** -126
