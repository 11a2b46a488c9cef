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
