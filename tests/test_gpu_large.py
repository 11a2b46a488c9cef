"""Sizes at the ends of the accepted ranges."""
import pytest
import torch

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    torch_cuda()
    import quantized_weight_decode_amd as q
    return q


def test_combine_of_more_tokens_than_a_launch(q):
    """2^24 tokens, a workgroup of 256 threads each: 2^32 work items, one more
    than a launch takes."""
    T, O, R = 1 << 24, 193, 5
    g = torch.Generator(device="cuda")
    g.manual_seed(80)
    h = torch.randn((R, O), dtype=torch.bfloat16, device="cuda", generator=g)
    pos = torch.randint(0, R, (T, 1), dtype=torch.int32, device="cuda", generator=g)
    gates = torch.rand((T, 1), device="cuda", generator=g)
    y = q.moe_combine(h, pos, gates)
    for lo in range(0, T, 1 << 21):
        hi = lo + (1 << 21)
        # one product: f32's rounding, then bf16's
        want = (h[pos[lo:hi, 0].long()].float() * gates[lo:hi]).to(torch.bfloat16)
        assert torch.equal(y[lo:hi], want)


def _exact_int4(O, I, g):
    """Weights (q - 8) / 8 and their values: products with whole x sum exactly."""
    w = torch.randint(0, 256, (O, I // 2), dtype=torch.uint8, device="cuda", generator=g)
    return w, torch.stack((w & 15, w >> 4), -1).reshape(O, I).to(torch.int8) - 8


def test_rows_too_long_to_pack(q):
    """I = 2^24: the packed rows of 128 tokens would take 4 GB; no scratch."""
    I, O, S, gs = 1 << 24, 3, 128, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(81)
    w, v = _exact_int4(O, I, g)
    s = torch.full((O, I // gs), 0.125, device="cuda")
    x = torch.randint(-1, 2, (S, I), dtype=torch.int8, device="cuda", generator=g)
    x = x.to(torch.bfloat16)
    y = q.i4g_linear(w, s, x, gs, residual=torch.zeros((S, O), device="cuda",
                                                       dtype=torch.bfloat16))
    want = torch.zeros((S, O), dtype=torch.float64, device="cuda")
    for lo in range(0, I, 1 << 20):
        k = slice(lo, lo + (1 << 20))
        want += torch.mm(x[:, k].double(), v[:, k].double().t().contiguous())
    # sums of whole eighths below 2^24 of them: exact, then one rounding
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(y, (want / 8).to(torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped_rows_of_more_tokens_than_can_be_packed(q, dtype):
    """Tokens whose packed rows exceed 4 GB, read through an index."""
    I, O, E, T, R, gs = 1 << 16, 40, 3, 33000, 90, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(82)
    w, v = _exact_int4(E * O, I, g)
    s = torch.full((E, O, I // gs), 0.125, device="cuda")
    x = torch.zeros((T, I), dtype=dtype, device="cuda")
    rows = torch.randint(T - 200, T, (R,), dtype=torch.int32, device="cuda", generator=g)
    x[T - 200:] = torch.randint(-1, 2, (200, I), device="cuda", generator=g).to(dtype)
    off = torch.tensor([0, 30, 31, R], dtype=torch.int32, device="cuda")
    y = q.i4g_grouped(w.view(E, O, I // 2), s, x, off, gs, rows=rows)
    for e, (lo, hi) in enumerate([(0, 30), (30, 31), (31, R)]):
        want = torch.mm(x[rows[lo:hi].long()].double(),
                        v[e * O:(e + 1) * O].double().t().contiguous()) / 8
        assert torch.equal(y[lo:hi], want.to(dtype))
