"""Inputs, 64-bit references and error bounds for the products with an
epilogue (not a test module).

Bound of one output.  The kernels form exact products of decoded weights and
activations (or activations split without loss to 2^-22 of themselves), sum
them in f32 and apply each scale to a group's f32 sum.  A sum of n terms of
total magnitude m, in any order, is off by at most n 2^-24 m (to first order);
scales, bias and the split add a few roundings: n = I + 16.  An activation of
slope below 1.13 passes that on, its own evaluation costs a few roundings of
its argument and value (16 2^-24 covers them), the gate multiplies, the
residual adds one rounding, and the result is rounded once to its type.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]


def int4(lead, I, gs, seed):
    r = np.random.default_rng(seed)
    w = r.integers(0, 256, (*lead, (I + 1) // 2), dtype=np.uint8)
    s = r.uniform(0.002, 0.02, (*lead, -(-I // gs))).astype(np.float32)
    return w, s


def fp8(O, I, seed):
    r = np.random.default_rng(seed)
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    w = codes[r.integers(0, 254, (O, I))]
    s = np.exp(r.uniform(np.log(1e-4), np.log(1e-2), (-(-O // 128), -(-I // 128))))
    return w, s.astype(np.float32)


def decode_int4(w, s, I, gs):
    q = np.stack([w & 15, w >> 4], -1).reshape(*w.shape[:-1], -1)[..., :I].astype(np.float64)
    return (q - 8.0) * np.repeat(s.astype(np.float64), gs, -1)[..., :I]


def decode_fp8(w, s):
    v = torch.from_numpy(w).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    sc = np.repeat(np.repeat(s.astype(np.float64), 128, 0), 128, 1)
    return v * sc[:w.shape[0], :w.shape[1]]


def acts(n, I, dtype, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn((n, I), generator=g).to(dtype)


def _act(a, act):
    if act == "relu":
        return torch.clamp_min(a, 0.0)
    if act == "silu":
        return a * torch.sigmoid(a)
    if act == "gelu":
        return 0.5 * a * torch.special.erfc(-a / 2.0 ** 0.5)
    if act == "gelu_tanh":
        return 0.5 * a * (1.0 + torch.tanh((2.0 / np.pi) ** 0.5 * (a + 0.044715 * a ** 3)))
    return a


def reference(W, x, dtype, bias=None, act=None, gated=False, residual=None):
    """(y, bound) in f64 for decoded W [O][I] (numpy f64) and x [S][I]."""
    W = torch.from_numpy(np.ascontiguousarray(W))
    x = x.cpu().double()
    n = W.shape[1] + 16
    a = x @ W.t()
    da = n * U * (x.abs() @ W.abs().t())
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


def assert_within(y, ref, bound, what=""):
    y = y.cpu().double()
    assert y.shape == ref.shape
    assert torch.isfinite(y).all(), f"{what}: {int((~torch.isfinite(y)).sum())} not finite"
    over = (y - ref).abs() / bound
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound at {int(over.argmax())}"


def rel_l2(y, ref):
    return float((y.cpu().double() - ref).norm() / ref.norm())
