"""Magnitudes of the products with an epilogue: rows and scales far from one,
few and many rows (the kernels that take them differ), against 64-bit
references within linear_util's bound.  All outputs are finite in their type,
and so are the sums of |x w|."""
import numpy as np
import pytest
import torch

import linear_util as L
from gpu_util import dev, torch_cuda

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.bfloat16]
# rows: the stream kernel with four rows, with 16, with 32 (bf16), the packed
# kernels, the same with wide tiles
ROWS = [(1, 300), (3, 300), (12, 300), (20, 9000), (60, 6100), (700, 1100)]


@pytest.fixture(scope="module")
def q():
    torch_cuda()
    import quantized_weight_decode_amd as q
    return q


def _weights(fmt, O, I, gs, seed):
    if fmt == "i4g":
        w, s = L.int4((O,), I, gs, seed)
        return w, s, lambda v: L.decode_int4(w, v, I, gs)
    w, s = L.fp8(O, I, seed)
    return w, s, lambda v: L.decode_fp8(w, v)


def _call(q, fmt, w, s, x, gs, **k):
    if fmt == "i4g":
        return q.i4g_linear(dev(w), dev(s), x.cuda(), gs, **k)
    return q.fp8b128_linear(dev(w), dev(s), x.cuda(), **k)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("fmt,gs", [("i4g", 32), ("i4g", 64), ("i4g", 128), ("fp8", 128)])
@pytest.mark.parametrize("S,O", ROWS)
def test_large_activations(q, fmt, gs, S, O, dtype):
    """Rows of one sign and of both up to 2^127, scales that bring the result
    back: no kernel overflows on the way."""
    I = 256
    w, s, decode = _weights(fmt, O, I, gs, 60)
    s = (s * np.float32(2.0 ** -40)).astype(np.float32)
    x = L.acts(S, I, torch.float32, 61).clamp(-3.9, 3.9)
    x[0::3] = x[0::3].abs() + 1.0
    x[0] = 1.9
    x = (x * 2.0 ** torch.tensor([119.0, 125.0, 112.0])[torch.arange(S) % 3][:, None]).to(dtype)
    x[0] *= 2.0 ** 7                                     # 1.9 * 2^126
    assert bool(torch.isfinite(x).all())
    ref, bound = L.reference(decode(s), x, dtype)
    L.assert_within(_call(q, fmt, w, s, x, gs), ref, bound)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("fmt,gs", [("i4g", 32), ("i4g", 64), ("i4g", 128), ("fp8", 128)])
@pytest.mark.parametrize("code", ["largest", "smallest", "zero"])
@pytest.mark.parametrize("S,O", ROWS)
def test_large_activations_times_extreme_codes(q, fmt, gs, S, O, code, dtype):
    """The largest group sums: all weights at one end, all of x one value."""
    I = 256
    nib = {"largest": 0x00, "smallest": 0x99, "zero": 0x88}[code]
    byte = {"largest": 0xFE, "smallest": 0x01, "zero": 0x00}[code]
    w, s, decode = _weights(fmt, O, I, gs, 62)
    w[:] = nib if fmt == "i4g" else byte
    s = (s * np.float32(2.0 ** -40)).astype(np.float32)
    x = torch.full((S, I), 1.9 * 2.0 ** 126, dtype=dtype)
    if S > 1:
        x[1, 0::2] *= -1
    ref, bound = L.reference(decode(s), x, dtype)
    L.assert_within(_call(q, fmt, w, s, x, gs), ref, bound)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("fmt", ["i4g", "fp8"])
@pytest.mark.parametrize("S,O", ROWS)
def test_large_scales(q, fmt, S, O, dtype):
    """Scales of 2^70 and small rows."""
    I, gs = 256, 64
    w, s, decode = _weights(fmt, O, I, gs, 63)
    s = (s * np.float32(2.0 ** 79)).astype(np.float32)
    x = (L.acts(S, I, torch.float32, 64) * 2.0 ** -60).to(dtype)
    ref, bound = L.reference(decode(s), x, dtype)
    L.assert_within(_call(q, fmt, w, s, x, gs), ref, bound)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("fmt", ["i4g", "fp8"])
@pytest.mark.parametrize("S,O", ROWS)
def test_small_activations(q, fmt, S, O, dtype):
    """Rows near 2^-100 with the outputs in the normal range: as exact as
    others."""
    I, gs = 256, 64
    w, s, decode = _weights(fmt, O, I, gs, 65)
    s = (s * np.float32(2.0 ** 60)).astype(np.float32)
    x = (L.acts(S, I, torch.float32, 66) * 2.0 ** -100).to(dtype)
    ref, bound = L.reference(decode(s), x, dtype)
    y = _call(q, fmt, w, s, x, gs)
    L.assert_within(y, ref, bound)
    if dtype == torch.float32:
        assert L.rel_l2(y, ref) <= 1e-5


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("counts", [[3, 0, 9, 1], [300, 5, 0, 411]])
def test_grouped_large_activations(q, counts, dtype):
    E, R, I, O, gs = len(counts), sum(counts), 256, 300, 64
    w, s = L.int4((E, O), I, gs, 67)
    s = (s * np.float32(2.0 ** -40)).astype(np.float32)
    x = (L.acts(R, I, torch.float32, 68).abs().clamp(0.5, 3.9) * 2.0 ** 125).to(dtype)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = q.i4g_grouped(dev(w), dev(s), x.cuda(), dev(off), gs)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            ref, bound = L.reference(L.decode_int4(w[e], s[e], I, gs), x[lo:hi], dtype)
            L.assert_within(y[lo:hi], ref, bound, f"expert {e}")


@pytest.mark.parametrize("fmt", ["i4g", "fp8"])
@pytest.mark.parametrize("S,O", [(1000, 4000), (500, 4000), (300, 1702), (100, 4200)])
@pytest.mark.parametrize("I,gs", [(160, 32), (256, 64), (96, 96), (448, 64)])
def test_f32_precision_of_the_packed_kernels(q, fmt, S, O, I, gs):
    """f32 x is packed to 22 bits at least.  Relative L2 over all outputs: the
    packing's errors, at most 2^-22 of an element and of either sign, give at
    most 2^-22; the sums' roundings, each at most 2^-24 of a partial sum of the
    output's size and of either sign, of N = I / 32 * 2 * 8 + I / 32 < 240 (two
    planes, each matrix instruction eight additions, one FMA per scale group)
    give sqrt(240) 2^-24 / sqrt(3) < 2^-20.8.  Together below 2^-20; twice that
    is asked.  x rounded to 16 bits would give 2^-16 sqrt(1/3) 0.7 = 2^-17.3.
    """
    w, s, decode = _weights(fmt, O, I, gs, 90)
    x = L.acts(S, I, torch.float32, 91)
    ref, _ = L.reference(decode(s), x, torch.float32)
    assert L.rel_l2(_call(q, fmt, w, s, x, gs), ref) <= 2.0 ** -19
