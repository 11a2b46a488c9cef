"""Operands in one buffer: those that share no element run as others do, those
that do are refused and leave the output as it was."""
import pytest
import torch

import linear_util as L
from gpu_util import dev, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    torch_cuda()
    import quantized_weight_decode_amd as q
    return q


@pytest.mark.parametrize("S", [1, 6, 40, 300])
def test_columns_of_one_buffer(q, S):
    """x, residual and y side by side in the rows of one buffer."""
    I, O, gs = 320, 90, 64
    w, s = L.int4((O,), I, gs, 70)
    buf = torch.zeros((S, I + 2 * O), dtype=torch.bfloat16, device="cuda")
    x, r = L.acts(S, I, torch.bfloat16, 71), L.acts(S, O, torch.bfloat16, 72)
    buf[:, :I], buf[:, I:I + O] = x.cuda(), r.cuda()
    out = buf[:, I + O:]
    q.i4g_linear(dev(w), dev(s), buf[:, :I], gs, residual=buf[:, I:I + O], out=out)
    ref, bound = L.reference(L.decode_int4(w, s, I, gs), x, torch.bfloat16, residual=r)
    L.assert_within(out, ref, bound)
    assert torch.equal(buf[:, :I].cpu(), x) and torch.equal(buf[:, I:I + O].cpu(), r)


def test_shared_elements_are_refused(q):
    I, gs = 64, 32
    w, s = (dev(t) for t in L.int4((I,), I, gs, 73))
    x = L.acts(20, I, torch.float32, 74).cuda()
    keep = x.clone()
    with pytest.raises(q.QgemvError, match="overlap"):
        q.i4g_linear(w, s, x, gs, out=x)
    with pytest.raises(q.QgemvError, match="overlap"):
        q.i4g_linear(w, s, x[:10], gs, out=x[9:19])
    with pytest.raises(q.QgemvError, match="overlap"):
        q.i4g_linear(w, s, x[:5].clone(), gs, residual=x[:5], out=x[1:6])
    pos = torch.zeros((20, 1), dtype=torch.int32, device="cuda")
    with pytest.raises(q.QgemvError, match="overlap"):
        q.moe_combine(x, pos, torch.ones((20, 1), device="cuda"), out=x)
    assert torch.equal(x, keep)
