"""8-bit products: the gradient of x by the transposed weights, dense, and operands
whose 32-bit offsets in the tile kernel pass 2^31."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from matmul_plan_util import plan
from matmul_util import (HALF, U, assert_within, decode_rows, decode_weights, reference, rows,
                         values, weights)

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


SIZES = [(1, 128, 256), (5, 300, 130), (70, 384, 1000), (150, 1000, 392), (300, 520, 7168)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S,I,O", SIZES)
def test_gradient_of_x(q, S, I, O, dtype):
    """dx = dy W: codes and scales transposed are W^T in the same format, so the last
    blocks of O are the last columns of the product."""
    w, s = weights((), O, I, 1)
    dy, ds = q.fp8_quantize(randn((S, O), 2).cuda())
    wt, st = cuda(w).t().contiguous(), cuda(s).t().contiguous()
    dx = q.fp8b128_matmul(wt, st, dy, ds, dtype=dtype)
    W = decode_weights(w, s)
    ref, bound = reference(np.ascontiguousarray(W.T), decode_rows(dy, ds), dtype)
    assert_within(dx, ref, bound)


@pytest.mark.parametrize("S,I,O", SIZES)
def test_gradient_of_x_by_differences(q, S, I, O):
    """<dy, y(a) - y(b)> = <dx, a - b> for the y of the forward product, f32: y is
    linear in x, so the difference has no error but the products' own."""
    w, s = weights((), O, I, 3)
    W = decode_weights(w, s)
    (a, sa), (b, sb) = rows(S, I, 4), rows(S, I, 5)
    dy, ds = q.fp8_quantize(randn((S, O), 6).cuda())
    wd, sd = cuda(w), cuda(s)
    ya, yb = (q.fp8b128_matmul(wd, sd, cuda(c), cuda(t), dtype=torch.float32).cpu().double()
              for c, t in ((a, sa), (b, sb)))
    dx = q.fp8b128_matmul(wd.t().contiguous(), sd.t().contiguous(), dy, ds,
                          dtype=torch.float32).cpu().double()
    g, xa, xb = decode_rows(dy, ds), decode_rows(a, sa), decode_rows(b, sb)
    num, ana = (g * (ya - yb)).sum(), (dx * (xa - xb)).sum()
    # every output is off by at most its bound
    _, ba = reference(W, xa, torch.float32)
    _, bb = reference(W, xb, torch.float32)
    _, bx = reference(np.ascontiguousarray(W.T), g, torch.float32)
    slack = (g.abs() * (ba + bb)).sum() + ((xa - xb).abs() * bx).sum()
    assert abs(num - ana) <= slack + 1e-9 * (abs(num) + abs(ana))


def need(gb):
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_x_behind_2_gb(q, dtype):
    """Grouped rows through an index, T * ldx between 2^31 and 2^32 bytes."""
    T, I, O, E = 65000, 65536, 264, 2
    assert 1 << 31 < T * I < 1 << 32
    need(12)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    x = torch.randint(0, 126, (T, I), dtype=torch.uint8, generator=g, device="cuda")
    xs = torch.rand((T, I // 128), generator=g, device="cuda")
    w, s = weights((E,), O, I, 8)
    pick = torch.tensor([T - 1, 0, 32767, 32768, T - 2, 40000, 1, 50001, 64998] * 5,
                        dtype=torch.int32)
    R = len(pick)
    assert plan(R, I, O, bf16=dtype == torch.bfloat16, E=E).tile
    offsets = torch.tensor([0, 20, R], dtype=torch.int32)
    y = q.fp8b128_matmul_grouped(cuda(w), cuda(s), x, xs, offsets.cuda(), rows=pick.cuda(),
                                 dtype=dtype)
    at = pick.long().cuda()
    xd = decode_rows(x[at], xs[at])
    for e, (lo, hi) in enumerate(((0, 20), (20, R))):
        ref, bound = reference(decode_weights(w[e], s[e]), xd[lo:hi], dtype)
        assert_within(y[lo:hi], ref, bound, f"expert {e}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_longest_rows(q, dtype):
    """256 rows of W and 70 of x with 2^24 - 16 columns, so that a tile's own offsets
    reach 2^32: nonzero weights at a few columns of each row only, in blocks of their
    own, so that every sum is of eight exact products."""
    S, I, O, n = 70, (1 << 24) - 16, 256, 8
    need(12)
    assert plan(S, I, O, bf16=dtype == torch.bfloat16).tile
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    # x from 2^-2 and weights from 1 up: no bit of a product lies below 2^-8, where the
    # zero weights' products (2^2 at most, by exponent) could cut it
    x = torch.randint(0x28, 126, (S, I), dtype=torch.uint8, generator=g, device="cuda")
    xs = torch.rand((S, -(-I // 128)), generator=g, device="cuda") + 0.5
    s = torch.rand((O // 128, -(-I // 128)), generator=g, device="cuda") + 0.5
    r = np.random.default_rng(10)
    # a column of each eighth of the row, the first and the last among them
    cols = (np.arange(n) * (I // n) + r.integers(0, I // n, (O, n))).astype(np.int64)
    cols[::3, 0], cols[1::3, n - 1] = 0, I - 1
    codes = (r.integers(0x38, 126, (O, n)) | r.integers(0, 2, (O, n)) << 7).astype(np.uint8)
    w = torch.zeros((O, I), dtype=torch.uint8, device="cuda")
    w.scatter_(1, cuda(cols), cuda(codes))
    y = q.fp8b128_matmul(w, s, x, xs, dtype=dtype).cpu().double()
    at = torch.from_numpy(cols)
    blocks = at // 128
    wv = torch.from_numpy(values(codes)) * s.cpu().double()[
        (torch.arange(O) // 128)[:, None], blocks]
    xh, xsh = x[:, at.reshape(-1).cuda()].cpu().numpy(), xs[:, blocks.reshape(-1).cuda()].cpu()
    terms = torch.from_numpy(values(xh)).reshape(S, O, n) * xsh.double().reshape(S, O, n) * wv
    ref, mag = terms.sum(2), terms.abs().sum(2)
    # one product per block: exact but for the scales' product and each addition
    bound = (2 * n + 2) * U * mag
    assert ((y - ref).abs() <= bound + HALF[dtype] * (ref.abs() + bound)).all()
