"""f32 operands whose rows lie on 16 bytes and not on 32: the widest loads and stores
ask for no more than 16."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from matmul_util import (assert_within, decode_rows, decode_weights, quantize, reference, rows,
                         weights)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    torch_cuda()
    import quantized_weight_decode_amd as q
    q.lib()
    return q


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def randn(shape, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(shape, generator=g)


def off(t, pad):
    """t's values, the first row 16 bytes behind a multiple of 32, rows `pad` elements
    longer; pad 4: every other row on 32 bytes, pad 8: none."""
    wide = torch.zeros(t.shape[0] * (t.shape[1] + pad) + 4, device="cuda")
    v = wide[4:].view(t.shape[0], -1)[:, :t.shape[1]]
    v.copy_(t)
    assert v.data_ptr() % 32 == 16
    return v


@pytest.mark.parametrize("pad", [4, 8])
@pytest.mark.parametrize("S,I", [(1, 128), (5, 384), (70, 1000)])
def test_quantizer(q, S, I, pad):
    x = randn((S, I), S + I)
    codes, scales = q.fp8_quantize(off(x, pad))
    want = quantize(x)
    assert np.array_equal(codes.cpu().numpy(), want[0])
    assert np.array_equal(scales.cpu().numpy(), want[1])


@pytest.mark.parametrize("pad", [4, 8])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("S,I,O", [(130, 384, 272), (300, 7168, 528)])
def test_product(q, S, I, O, gated, pad):
    """y, residual and bias; the second size also with parts of K."""
    w, s = weights((), O, I, 1)
    c, cs = rows(S, I, 2)
    oc = O // 2 if gated else O
    bias, res = randn((O,), 3), randn((S, oc), 4)
    ref, bound = reference(decode_weights(w, s), decode_rows(c, cs), torch.float32, bias,
                           "silu", gated, res)
    args = [cuda(t) for t in (w, s, c, cs)]
    b = off(bias[None], 0)[0]
    out = off(torch.zeros((S, oc)), pad)
    q.fp8b128_matmul(*args, bias=b, act="silu", gated=gated, residual=off(res, pad), out=out)
    assert_within(out, ref, bound)
    alone = q.fp8b128_matmul(*args, bias=bias.cuda(), act="silu", gated=gated,
                             residual=res.cuda())
    assert torch.equal(out, alone)


@pytest.mark.parametrize("pad", [4, 8])
@pytest.mark.parametrize("S", [20, 300])
def test_many_token_product_with_f32_rows(q, S, pad):
    I, O = 512, 256
    w, s = weights((), O, I, 5)
    x = randn((S, I), 6)
    args = cuda(w), cuda(s)
    assert torch.equal(q.fp8b128_linear(*args, off(x, pad)), q.fp8b128_linear(*args, x.cuda()))
