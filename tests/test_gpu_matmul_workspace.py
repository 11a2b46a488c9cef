"""Scratch of the 8-bit products for calls of several numbers of rows."""
import numpy as np
import pytest
import torch

from matmul_util import rows, weights

I, O = 7168, 7176


@pytest.fixture(scope="module")
def q():
    import quantized_weight_decode_amd as q
    try:
        q.lib()
    except ImportError as e:
        pytest.skip(str(e))
    return q


def test_of_other_rows_is_refused_by_name(q):
    """What the most rows need is not a bound for fewer: it has to be asked for each
    S, and too little is refused before anything runs."""
    need = {S: q.qgemv_matmul_workspace(S, I, O, 1, 0) for S in range(1, 2049)}
    assert all(n % 256 == 0 for n in need.values())
    fewer = max(need, key=need.get)
    more = next(S for S in range(fewer + 1, 2049) if need[S] < need[fewer])
    A = 1 << 40                                 # operands far apart, never read
    st = q.qgemv_fp8b128_matmul(A, 2 * A, 3 * A, I, 4 * A, 56, 5 * A, O, fewer, I, O, 1, None,
                                7 * A, need[more], 0)
    assert st == 7, need[more]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gated", [False, True])
def test_the_largest_of_several_serves_them_all(q, dtype, gated):
    def cuda(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()
    w, s = (cuda(t) for t in weights((), O, I, 1))
    sizes = [4, 40, 70, 300, 500, 1100]
    each = [q.matmul_workspace(S, I, O, dtype, "cuda", gated) for S in sizes]
    assert max(t.numel() for t in each[:-1]) > each[-1].numel()
    ws = max(each, key=torch.Tensor.numel).fill_(0x5A)
    for S, own in zip(sizes, each):
        x, xs = (cuda(t) for t in rows(S, I, S))
        want = q.fp8b128_matmul(w, s, x, xs, gated=gated, dtype=dtype)
        for scratch in (ws, own):
            y = q.fp8b128_matmul(w, s, x, xs, gated=gated, dtype=dtype, workspace=scratch)
            assert torch.equal(y, want)
