"""Every way that the tile kernel takes a dense bfloat16 product: kinds of tiles, parts
of K, a launch of their own for the first columns, and these together."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from matmul_plan_util import REACHED, plan
from matmul_util import assert_within, decode_rows, decode_weights, reference, rows, weights

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
    return torch.randn(shape, generator=g).bfloat16()


def one_of_16(n, r):
    """An index of each 16 consecutive ones, the first and the last."""
    at = np.arange(0, n, 16)
    return np.unique(np.concatenate([np.minimum(at + r.integers(0, 16, len(at)), n - 1),
                                     [0, n - 1]]))


@pytest.mark.parametrize("kind,cut,head,S,I,O,gated", REACHED)
def test_every_plan(q, kind, cut, head, S, I, O, gated):
    """A row of each 16 over all columns, and a column of each 16 over all rows: every
    fragment of every tile, and the columns where launches and tiles meet."""
    ncu = torch.cuda.get_device_properties(0).multi_processor_count
    p = plan(S, I, O, gated=gated, ncu=ncu)
    assert p.tile and p.kind == kind and (p.parts > 1) == cut
    assert (p.head_kind if p.head else None) == head
    oc = O // 2 if gated else O
    w, s = weights((), O, I, S)
    c, cs = rows(S, I, S + 1)
    bias, res = randn((O,), S + 2), randn((S, oc), S + 3)
    act = "silu" if gated else "relu"
    need = q.qgemv_matmul_workspace(S, I, O, 1, int(gated))
    assert (need > 0) == cut
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    buf = torch.full((S + 2, oc), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:S + 1]
    q.fp8b128_matmul(cuda(w), cuda(s), cuda(c), cuda(cs), bias=bias.cuda(), act=act, gated=gated,
                     residual=res.cuda(), out=out, workspace=ws[:need] if need else None)
    assert (ws[need:] == 0x5A).all() and (buf[0] == 7.0).all() and (buf[-1] == 7.0).all()
    y, r = out.cpu(), np.random.default_rng(S)
    W, x = decode_weights(w, s), decode_rows(c, cs)
    some = one_of_16(S, r)
    ref, bound = reference(W, x[some], torch.bfloat16, bias, act, gated, res[some])
    assert_within(y[some], ref, bound, "rows")
    some = one_of_16(oc, r)
    both = np.concatenate([some, some + oc]) if gated else some
    ref, bound = reference(W[both], x, torch.bfloat16, bias[both], act, gated, res[:, some])
    assert_within(y[:, some], ref, bound, "columns")
