"""Activations in 8 bits: codes and scales bit for bit against the definition."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from matmul_util import FINITE, quantize

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    torch_cuda()
    import quantized_weight_decode_amd as q
    q.lib()
    return q


def same(got, want):
    codes, scales = got
    assert np.array_equal(scales.cpu().numpy(), want[1], equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), want[0])


def randn(S, I, dtype, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    # rows of very different magnitude
    return (torch.randn((S, I), generator=g) * torch.exp(3 * torch.randn((S, 1), generator=g))
            ).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S,I", [(1, 1), (1, 128), (3, 7), (4, 7168), (7, 129), (33, 1000),
                                 (130, 2040), (513, 264), (5, 16385)])
def test_random(q, S, I, dtype):
    x = randn(S, I, dtype, S + I)
    same(q.fp8_quantize(x.cuda()), quantize(x))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_borders(q, dtype):
    """Every code, the values half way between two and their neighbours, at scales
    that are exact: 448 times a power of two in each block."""
    v = np.unique(np.abs(torch.from_numpy(FINITE).view(torch.float8_e4m3fn).double().numpy()))
    mid = (v[1:] + v[:-1]) / 2
    t = np.concatenate([v, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20), v * 1.01])
    t = np.concatenate([t, -t])
    t = t[np.abs(t) <= 448]
    t = np.resize(t, (-(-len(t) // 127) * 127,)).reshape(-1, 127)
    x = np.concatenate([np.full((len(t), 1), 448.0), t], 1)
    for e in (-100, -9, 0, 5, 100):
        xe = torch.from_numpy(x * 2.0 ** e).to(dtype)
        same(q.fp8_quantize(xe.cuda()), quantize(xe))


def test_quotients_next_to_the_middle_of_two_codes(q):
    """x as near to middle * max / 448 as f32 gets, and its neighbours: an f32 quotient
    of an f32 scale would put some of them on the wrong side."""
    r = np.random.default_rng(7)
    v = np.unique(np.abs(torch.from_numpy(FINITE).view(torch.float8_e4m3fn).double().numpy()))
    mid = np.resize((v[1:] + v[:-1]) / 2, 127)
    top = (r.uniform(1, 2, (600, 1)) * np.exp2(r.integers(-60, 60, (600, 1)))).astype(np.float32)
    x = (mid * top.astype(np.float64) / 448).astype(np.float32)
    for k in (0, -1, 1):
        near = x if k == 0 else np.nextafter(x, np.float32(k) * np.inf, dtype=np.float32)
        t = torch.from_numpy(np.concatenate([top, near * np.where(r.random(near.shape) < 0.5, -1, 1)
                                             .astype(np.float32)], 1))
        same(q.fp8_quantize(t.cuda()), quantize(t))
    # bfloat16, whose quotients hit middles exactly: 0.75 of the largest and its like
    top = torch.from_numpy(r.uniform(1, 2, (2000, 1))).bfloat16()
    t = torch.cat([top, (top.float() * torch.from_numpy(np.resize(mid, (1, 127))).float() / 448)
                   .bfloat16()], 1)
    same(q.fp8_quantize(t.cuda()), quantize(t))


def test_smallest_and_largest(q):
    rows = [np.zeros(256), np.full(256, 2.0 ** -149), np.full(256, -2.0 ** -126),
            np.linspace(-1, 1, 256) * 2.0 ** -118, np.linspace(-1, 1, 256) * 2.0 ** -117.3,
            np.linspace(-1, 1, 256) * 3.4e38, np.full(256, -0.0),
            np.where(np.arange(256) == 200, 3.4e38, 1e-30)]
    x = torch.from_numpy(np.stack(rows)).float()
    same(q.fp8_quantize(x.cuda()), quantize(x))
    b = x.bfloat16()
    same(q.fp8_quantize(b.cuda()), quantize(b))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinity_and_nan_poison_their_block(q, dtype):
    x = randn(6, 300, dtype, 3)
    x[1, 5] = float("inf")
    x[2, 299] = float("nan")
    x[4, 128] = -float("inf")
    codes, scales = q.fp8_quantize(x.cuda())
    clean = x.clone()
    clean[1, :128] = clean[2, 256:] = clean[4, 128:256] = 0.0
    want_c, want_s = quantize(clean)
    want_c[1, :128] = want_c[2, 256:] = want_c[4, 128:256] = 0x7F
    want_s[1, 0] = want_s[2, 2] = want_s[4, 1] = np.nan
    assert np.array_equal(scales.cpu().numpy(), want_s, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), want_c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off,pad", [(0, 8), (1, 3), (4, 4), (3, 13)])
def test_strides_and_what_is_left(q, dtype, off, pad):
    S, I = 9, 391
    x = randn(S, I, dtype, 4)
    wide = torch.zeros((S, I + pad + off), dtype=dtype, device="cuda")
    xv = wide[:, off:off + I]
    xv.copy_(x)
    cb = torch.full((S, I + pad + off), 0x55, dtype=torch.uint8, device="cuda")
    sb = torch.full((S, 4 + pad), -1.0, device="cuda")
    codes, scales = q.fp8_quantize(xv, out=cb[:, off:off + I], scales=sb[:, 1:5])
    same((codes, scales), quantize(x))
    codes.fill_(0x55)
    scales.fill_(-1.0)
    assert (cb == 0x55).all() and (sb == -1.0).all()
    one = q.fp8_quantize(x[2].cuda())
    assert one[0].shape == (I,) and one[1].shape == (4,)
    want = quantize(x[2:3])
    same((one[0][None], one[1][None]), want)


def test_no_rows_and_float8_out(q):
    c, s = q.fp8_quantize(torch.empty((0, 256), device="cuda"))
    assert c.shape == (0, 256) and s.shape == (0, 2)
    x = randn(3, 256, torch.float32, 5)
    out = torch.empty((3, 256), dtype=torch.float8_e4m3fn, device="cuda")
    got, s = q.fp8_quantize(x.cuda(), out=out)
    assert got is out
    want = quantize(x)
    assert np.array_equal(out.view(torch.uint8).cpu().numpy(), want[0])
