"""Token rows in expert order, their gradient, and the gradient of the experts'
return, against 64 bits; the whole routed layer forward and back."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from matmul_util import HALF, U, decode_rows, decode_weights, sum_bound, weights

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def q():
    torch_cuda()
    import quantized_weight_decode_amd as q
    q.lib()
    return q


def randn(shape, dtype, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def plan(q, T, K, E, seed, bad=0.0):
    r = np.random.default_rng(seed)
    ids = np.stack([r.choice(E, K, replace=False) for _ in range(T)]).astype(np.int32)
    ids[r.random((T, K)) < bad] = -1
    return q.moe_group(torch.from_numpy(ids).cuda(), E)


SIZES = [(1, 1, 2, 1), (5, 2, 4, 7), (33, 8, 64, 256), (70, 3, 9, 1030), (300, 6, 16, 2056),
         (17, 40, 64, 320), (9, 64, 100, 96)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,E,I", SIZES)
@pytest.mark.parametrize("pad", [0, 5])
def test_dispatch_and_its_gradient(q, T, K, E, I, dtype, pad):
    offsets, tokens, pos = plan(q, T, K, E, T + K, bad=0.1)
    x = randn((T, I + pad), dtype, 1).cuda()[:, :I]
    buf = torch.full((T * K, I + pad), 3.0, dtype=dtype, device="cuda")
    y = q.moe_dispatch(x, tokens, out=buf[:, :I])
    tok = tokens.cpu().long()
    want = torch.where((tok >= 0)[:, None], x.cpu()[tok.clamp_min(0)], torch.tensor(3.0).to(dtype))
    assert torch.equal(y.cpu(), want)
    assert (buf[:, I:] == 3.0).all()

    dy = randn((T * K, I + pad), dtype, 2).cuda()[:, :I]
    dx = q.moe_dispatch_grad(dy, pos)
    p = pos.cpu().long()
    rows = dy.cpu().double()[p.clamp_min(0)] * (p >= 0)[:, :, None]
    ref = rows.sum(1)
    bound = K * U * rows.abs().sum(1)
    bound = bound + HALF[dtype] * (ref.abs() + bound)
    assert ((dx.cpu().double() - ref).abs() <= bound).all()
    # <dispatch(x), dy> = <x, dispatch_grad(dy)>: the two are transposes
    valid = tok >= 0
    lhs = (x.cpu().double()[tok[valid]] * dy.cpu().double()[valid]).sum()
    rhs = (x.cpu().double() * dx.cpu().double()).sum()
    assert abs(lhs - rhs) <= (x.cpu().double().abs() * bound).sum() + 1e-9 * abs(lhs)


@pytest.mark.parametrize("dtype", TYPES)
def test_dispatch_bad_indices(q, dtype):
    x = randn((4, 40), dtype, 3).cuda()
    tokens = torch.tensor([3, -1, 4, 0, -2, 1 << 30, -(1 << 31), 3], dtype=torch.int32).cuda()
    y = q.moe_dispatch(x, tokens, out=torch.full((8, 40), 9.0, dtype=dtype, device="cuda"))
    for r, t in ((0, 3), (3, 0), (7, 3)):
        assert torch.equal(y[r], x[t])
    assert (y[1] == 9.0).all()
    assert y[[2, 4, 5, 6]].isnan().all()
    pos = torch.tensor([[0, 1], [-1, -1], [2, 8], [-2, 3], [4, 4]], dtype=torch.int32).cuda()
    dy = randn((8, 40), dtype, 4).cuda()
    dx = q.moe_dispatch_grad(dy, pos)
    assert dx[[2, 3]].isnan().all() and not dx[1].any()
    assert torch.equal(dx[0], (dy[0].float() + dy[1].float()).to(dtype))
    assert torch.equal(dx[4], (dy[4].float() + dy[4].float()).to(dtype))
    none = q.moe_dispatch_grad(dy[:0], torch.full((3, 2), -1, dtype=torch.int32, device="cuda"))
    assert none.shape == (3, 40) and not none.any()
    assert q.moe_dispatch(x, tokens[:0]).shape == (0, 40)


def combine_reference(dy, h, tokens, pos, gates):
    """(dh, rows written, dgates, bound of dgates) in f64."""
    T, K = pos.shape
    R, O = h.shape
    dy, h, gates = dy.cpu().double(), h.cpu().double(), gates.cpu().double()
    dh, wrote = torch.zeros((R, O), dtype=torch.float64), torch.zeros(R, dtype=torch.bool)
    dg, bound = torch.full((T, K), float("nan"), dtype=torch.float64), torch.zeros(T, K).double()
    for t in range(T):
        for k in range(K):
            p = int(pos[t, k])
            if 0 <= p < R and int(tokens[p]) == t:
                dh[p] += gates[t, k] * dy[t]
                wrote[p] = True
                dg[t, k] = (h[p] * dy[t]).sum()
                bound[t, k] = (O + 8) * U * (h[p] * dy[t]).abs().sum()
    return dh, wrote, dg, bound


def check_combine(q, dy, h, tokens, pos, gates, dtype, pad=0):
    R, O = h.shape
    buf = torch.full((R, O + pad), 4.0, dtype=dtype, device="cuda")
    dh, dg = q.moe_combine_grad(dy, h, tokens, pos, gates, out=buf[:, :O])
    ref, wrote, rg, bound = combine_reference(dy, h, tokens.cpu(), pos.cpu(), gates)
    got = dh.cpu().double()
    assert (got[~wrote] == 4.0).all() and (buf[:, O:] == 4.0).all()
    # gates of one row's slots summed (K 2^-24), one product, one rounding
    tol = (HALF[dtype] + (pos.shape[1] + 1) * U) * ref.abs() * 1.01 + 2.0 ** -126
    assert ((got - ref).abs() <= tol)[wrote].all()
    g = dg.cpu().double()
    assert torch.equal(g.isnan(), rg.isnan())
    ok = ~rg.isnan()
    assert ((g - rg).abs() <= bound + U * rg.abs())[ok].all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,E,O", SIZES)
@pytest.mark.parametrize("pad", [0, 5])
def test_combine_gradient(q, T, K, E, O, dtype, pad):
    offsets, tokens, pos = plan(q, T, K, E, 2 * T + K, bad=0.05)
    dy = randn((T, O + pad), dtype, 5).cuda()[:, :O]
    h = randn((T * K, O + pad), dtype, 6).cuda()[:, :O]
    gates = torch.softmax(randn((T, K), torch.float32, 7), 1).cuda()
    check_combine(q, dy, h, tokens, pos, gates, dtype, pad)


@pytest.mark.parametrize("dtype", TYPES)
def test_combine_gradient_of_shared_and_foreign_rows(q, dtype):
    """Two slots of a token on one row add their gates; a slot on another token's row
    or outside gets a NaN and writes none."""
    pos = torch.tensor([[0, 0, 1], [2, 1, 3], [9, -1, 4], [5, 5, 5]], dtype=torch.int32)
    tokens = torch.tensor([0, 0, 1, 3, 2, 3, -1], dtype=torch.int32)
    dy, h = randn((4, 130), dtype, 8).cuda(), randn((7, 130), dtype, 9).cuda()
    gates = randn((4, 3), torch.float32, 10).cuda()
    check_combine(q, dy, h, tokens.cuda(), pos.cuda(), gates, dtype)


def test_combine_gradient_by_differences(q):
    """d<y, dy> along a direction of h and of the gates, through moe_combine itself
    (f32; y is linear in each, so a difference has no error of its own beyond
    the roundings)."""
    T, K, E, O = 20, 4, 10, 200
    offsets, tokens, pos = plan(q, T, K, E, 11)
    h, dh = randn((T * K, O), torch.float32, 12).cuda(), randn((T * K, O), torch.float32, 13).cuda()
    g = torch.softmax(randn((T, K), torch.float32, 14), 1).cuda()
    dg = randn((T, K), torch.float32, 15).cuda()
    dy = randn((T, O), torch.float32, 16).cuda()

    def loss(h, g):
        return float((q.moe_combine(h, pos, g).double() * dy.double()).sum())
    gh, gg = q.moe_combine_grad(dy, h, tokens, pos, g)
    num = loss(h + dh, g) - loss(h - dh, g)
    ana = 2.0 * float((gh.double() * dh.double()).sum())
    size = float((h.abs().sum() + dh.abs().sum()))
    assert abs(num - ana) <= 2.0 ** -18 * size
    num = loss(h, g + dg) - loss(h, g - dg)
    ana = 2.0 * float((gg.double() * dg.double()).sum())
    assert abs(num - ana) <= 2.0 ** -18 * size * 4


def test_gradient_calls_replayed(q):
    T, K, E, O = 60, 4, 12, 520
    _, tokens, pos = plan(q, T, K, E, 17)
    sets = [(randn((T, O), torch.bfloat16, 18 + i).cuda(),
             randn((T * K, O), torch.bfloat16, 28 + i).cuda(),
             torch.softmax(randn((T, K), torch.float32, 38 + i), 1).cuda()) for i in range(3)]

    def calls(dy, h, g):
        return (*q.moe_combine_grad(dy, h, tokens, pos, g), q.moe_dispatch(dy, tokens),
                q.moe_dispatch_grad(h, pos), *q.fp8_quantize(h))
    alone = [tuple(t.clone() for t in calls(*v)) for v in sets]
    fixed = [t.clone() for t in sets[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(*fixed)
    for i in (1, 2, 0, 1):
        for t, v in zip(fixed, sets[i]):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(got, alone[i]):
            assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [3, 150])
def test_routed_layer_forward_and_back(q, T, dtype):
    """Router, sort, quantized gate and up projections, quantized down projection,
    return; then the gradients of the gates, of the experts' outputs, through the
    down projection's transpose, and of the sorted rows back to their tokens.
    Each step against 64 bits on its own inputs."""
    E, K, I, F = 8, 2, 256, 192
    x = randn((T, I), dtype, 20).cuda()
    logits = randn((T, E), torch.float32, 21).cuda()
    w1, s1 = weights((E,), 2 * F, I, 22)
    w2, s2 = weights((E,), I, F, 23)
    cu = [torch.from_numpy(t).cuda() for t in (w1, s1, w2, s2)]
    ids, gates = q.router_topk(logits, E, K)
    offsets, tokens, pos = q.moe_group(ids, E)
    xq, xs = q.fp8_quantize(x)
    h = q.fp8b128_matmul_grouped(cu[0], cu[1], xq, xs, offsets, rows=tokens, act="silu",
                                 gated=True, dtype=dtype)
    hq, hs = q.fp8_quantize(h)
    o = q.fp8b128_matmul_grouped(cu[2], cu[3], hq, hs, offsets, dtype=dtype)
    y = q.moe_combine(o, pos, gates, residual=x)

    off, tok = offsets.tolist(), tokens.cpu().long()
    W1, W2 = decode_weights(w1, s1), decode_weights(w2, s2)

    def product(W, rows):
        a, m = [], []
        for e in range(E):
            we = torch.from_numpy(W[e])
            r = rows[off[e]:off[e + 1]]
            a.append(r @ we.t())
            m.append(sum_bound(W[e], r, dtype))
        return torch.cat(a), torch.cat(m)
    a, da = product(W1, decode_rows(xq, xs)[tok])
    gate, up = a[:, :F], a[:, F:]
    ref = gate * torch.sigmoid(gate) * up
    d = (1.13 * da[:, :F] + 16 * U * gate.abs()) * (up.abs() + da[:, F:]) + gate.abs() * da[:, F:]
    d = d + (HALF[dtype] + 4 * U) * (ref.abs() + d)
    assert ((h.cpu().double() - ref).abs() <= d).all()
    ref, d = product(W2, decode_rows(hq, hs))
    d = d + HALF[dtype] * (ref.abs() + d)
    assert ((o.cpu().double() - ref).abs() <= d).all()

    dy = randn((T, I), dtype, 24).cuda()
    do, dgates = q.moe_combine_grad(dy, o, tokens, pos, gates)
    rdo, wrote, rdg, bound = combine_reference(dy, o, tok, pos.cpu(), gates)
    assert wrote.all()
    assert ((do.cpu().double() - rdo).abs() <= (HALF[dtype] + 4 * U) * rdo.abs() + 1e-37).all()
    assert ((dgates.cpu().double() - rdg).abs() <= bound + U * rdg.abs()).all()
    # dh = do W2 through the transposed codes, which are W2^T in the same format
    w2t, s2t = cu[2].transpose(1, 2).contiguous(), cu[3].transpose(1, 2).contiguous()
    dq, ds = q.fp8_quantize(do)
    dh = q.fp8b128_matmul_grouped(w2t, s2t, dq, ds, offsets, dtype=dtype)
    W2t = np.ascontiguousarray(W2.transpose(0, 2, 1))
    ref, d = product(W2t, decode_rows(dq, ds))
    d = d + HALF[dtype] * (ref.abs() + d)
    assert ((dh.cpu().double() - ref).abs() <= d).all()
    # what quantizing do added, against the product of the f64 gradient: each element
    # of do is within 2^-4 of itself or 2^-10 of its block's scale
    full, _ = product(W2t, do.cpu().double())
    mag, _ = product(np.abs(W2t), do.cpu().double().abs())
    steps = torch.repeat_interleave(ds.cpu().double(), 128, 1)[:, :I] * 2.0 ** -10
    slack = 2.0 ** -4 * mag + torch.cat([steps[off[e]:off[e + 1]] @ torch.from_numpy(
        np.abs(W2[e])) for e in range(E)])
    assert ((dh.cpu().double() - full).abs() <= slack + d + 4 * U * mag).all()
    dx = q.moe_dispatch_grad(dh, pos)
    assert dx.shape == (T, F) and torch.isfinite(dx.float()).all()
    want = dh.cpu().double()[pos.cpu().long()].sum(1)
    assert ((dx.cpu().double() - want).abs() <= (HALF[dtype] + 4 * U) *
            dh.cpu().double().abs()[pos.cpu().long()].sum(1)).all()
