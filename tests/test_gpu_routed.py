"""Routed slots sorted by expert, the grouped product and the return to the
tokens, on the GPU: one by one and as a routed MLP."""
import numpy as np
import pytest
import torch

import linear_util as L
from gpu_util import dev, torch_cuda

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def q():
    torch_cuda()
    import quantized_weight_decode_amd as q
    return q


def group_ref(ids, E):
    T, K = ids.shape
    rows = [[] for _ in range(E)]
    for i, e in enumerate(ids.reshape(-1)):
        if 0 <= e < E:
            rows[e].append(i)
    order = [i for r in rows for i in r]
    offsets = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int32)
    tokens = np.full(T * K, -1, np.int32)
    pos = np.full(T * K, -1, np.int32)
    for r, i in enumerate(order):
        tokens[r], pos[i] = i // K, r
    return offsets, tokens, pos.reshape(T, K)


@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (4, 8, 256), (3, 5, 7), (63, 1, 2), (200, 8, 1024),
                                   (256, 8, 64), (257, 8, 64), (2049, 1, 1), (3000, 7, 300),
                                   (65536, 9, 33)])
@pytest.mark.parametrize("law", ["even", "one", "invalid"])
def test_group(q, T, K, E, law):
    r = np.random.default_rng(T + E)
    ids = r.integers(0, E, (T, K)).astype(np.int32)
    if law == "one":
        ids[:] = E - 1
    if law == "invalid":
        ids = r.integers(-2, E + 2, (T, K)).astype(np.int32)
        ids.reshape(-1)[::11] = np.int32(-2 ** 31)
        ids.reshape(-1)[5::13] = np.int32(2 ** 31 - 1)
    for _ in range(2):
        got = q.moe_group(dev(ids), E)
        for g, w in zip(got, group_ref(ids, E)):
            assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w)


def test_group_without_tokens(q):
    o, t, p = q.moe_group(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 6)
    assert o.tolist() == [0] * 7 and t.numel() == 0 and p.shape == (0, 4)


def counts_offsets(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)


# row counts per expert: none, one, both sides of the tiles' rows
COUNTS = [[1], [0, 0, 1, 0], [3, 0, 16, 17, 1, 0], [64, 1, 65, 0, 31, 33], [128, 129, 0, 127],
          [300, 5], [1] * 40, [2, 0, 1, 3] * 16]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("I,O,gs", [(256, 96, 64), (101, 35, 6), (544, 258, 32)])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(q, counts, I, O, gs, gather, dtype):
    E, R = len(counts), int(np.sum(counts))
    w, s = L.int4((E, O), I, gs, R + I)
    off = counts_offsets(counts)
    r = np.random.default_rng(1)
    T = 9 if gather else R
    x = L.acts(T, I, dtype, 2)
    rows = r.integers(0, T, R).astype(np.int32) if gather else None
    bias = L.acts(E, O, dtype, 3)
    y = q.i4g_grouped(dev(w), dev(s), x.cuda(), dev(off), gs,
                      rows=dev(rows) if gather else None, bias=bias.cuda(), act="relu")
    xs = x[torch.from_numpy(rows).long()] if gather else x
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            ref, bound = L.reference(L.decode_int4(w[e], s[e], I, gs), xs[lo:hi], dtype,
                                     bias=bias[e], act="relu")
            L.assert_within(y[lo:hi], ref, bound, f"expert {e}")


@pytest.mark.parametrize("counts", [[3, 0, 2], [70, 140, 1]])
def test_grouped_rows_of_no_expert_stay(q, counts):
    """Rows before the first and behind the last expert keep their values, as
    do the columns beside out; R rows in all."""
    E, I, O, gs = 3, 128, 40, 32
    w, s = L.int4((E, O), I, gs, 4)
    off = counts_offsets(counts, first=5)
    R = int(off[-1]) + 9
    x = L.acts(R, I, torch.bfloat16, 5)
    buf = torch.full((R, O // 2 + 3), -3.0, dtype=torch.bfloat16, device="cuda")
    q.i4g_grouped(dev(w), dev(s), x.cuda(), dev(off), gs, act="silu", gated=True,
                  out=buf[:, 1:1 + O // 2])
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            ref, bound = L.reference(L.decode_int4(w[e], s[e], I, gs), x[lo:hi], torch.bfloat16,
                                     act="silu", gated=True)
            L.assert_within(buf[lo:hi, 1:1 + O // 2], ref, bound)
    buf[5:off[-1], 1:1 + O // 2] = -3.0
    assert bool((buf == -3.0).all())


def test_grouped_bad_row_index_gives_nan(q):
    E, I, O, gs = 2, 64, 24, 32
    w, s = L.int4((E, O), I, gs, 6)
    for n in (4, 80):
        off = counts_offsets([n, n])
        rows = np.zeros(2 * n, np.int32)
        rows[1], rows[n + 2] = -1, 3
        x = L.acts(3, I, torch.bfloat16, 7)
        y = q.i4g_grouped(dev(w), dev(s), x.cuda(), dev(off), gs, rows=dev(rows))
        bad = torch.isnan(y).cpu()
        assert bool(bad[1].all()) and bool(bad[n + 2].all())
        assert int(bad.sum()) == 2 * O


def test_grouped_odd_offsets_stay_inside(q):
    """Offsets that decrease or leave 0..R touch nothing outside y."""
    E, I, O, gs, R = 4, 64, 24, 32, 50
    w, s = L.int4((E, O), I, gs, 8)
    x = L.acts(R, I, torch.float32, 9).cuda()
    buf = torch.full((R + 200, O), 2.25, device="cuda")
    for off in ([-7, 3, 90, 20, 60], [50, 40, 30, 20, 10], [2 ** 31 - 1, -2 ** 31, 0, 50, 99]):
        q.i4g_grouped(dev(w), dev(s), x, dev(np.array(off, np.int64).astype(np.int32)), gs,
                      out=buf[100:100 + R])
        assert bool((buf[:100] == 2.25).all()) and bool((buf[100 + R:] == 2.25).all())


def test_grouped_expert_stack_beyond_32_bit_offsets(q):
    """The last expert's weights start past 4 GiB."""
    E, I, O, gs = 5, 64, 40, 32
    w, s = L.int4((E, O), I, gs, 10)
    stride = 1152 << 20
    buf = torch.empty((E - 1) * stride + O * I // 2, dtype=torch.uint8, device="cuda")
    for e in range(E):
        buf[e * stride:e * stride + O * I // 2] = dev(w[e]).reshape(-1)
    sd = dev(s)
    x = L.acts(40, I, torch.float32, 11)
    off = dev(counts_offsets([8] * E))
    y = torch.zeros((40, O), device="cuda")
    ws = q.grouped_workspace(40, 40, E, I, O, torch.float32, "cuda")
    xd = x.cuda()
    st = q.qgemv_i4g_grouped(buf.data_ptr(), sd.data_ptr(), stride, O * 2, E, off.data_ptr(), None,
                             xd.data_ptr(), I, 40, y.data_ptr(), O, 40, I, O, gs, 0, None,
                             ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for e in range(E):
        ref, bound = L.reference(L.decode_int4(w[e], s[e], I, gs), x[8 * e:8 * e + 8],
                                 torch.float32)
        L.assert_within(y[8 * e:8 * e + 8], ref, bound)


def combine_ref(h, pos, gates, dtype, residual=None):
    """(y, bound): K products and sums in f32, one rounding of the result."""
    hd = h.cpu().double()[pos.cpu().long()]
    g = gates.cpu().double()[:, :, None]
    y = (hd * g).sum(1)
    d = (pos.shape[1] + 1) * L.U * (hd * g).abs().sum(1)
    if residual is not None:
        y = y + residual.cpu().double()
        d = d + L.U * (y.abs() + d)
    return y, d + L.HALF[dtype] * (y.abs() + d) + 2.0 ** -126


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,K,O", [(1, 1, 1), (4, 8, 2048), (5, 3, 77), (33, 9, 64),
                                   (130, 64, 520), (700, 2, 1031)])
def test_combine(q, T, K, O, residual, dtype):
    r = np.random.default_rng(T + O)
    R = T * K + 3
    h = L.acts(R, O, dtype, 1)
    pos = torch.from_numpy(r.integers(0, R, (T, K)).astype(np.int32))
    gates = torch.from_numpy(r.dirichlet(np.ones(K), T).astype(np.float32))
    res = L.acts(T, O, dtype, 2) if residual else None
    y = q.moe_combine(h.cuda(), pos.cuda(), gates.cuda(),
                      residual=res.cuda() if residual else None)
    L.assert_within(y, *combine_ref(h, pos, gates, dtype, res))


def test_combine_bad_positions_strides_and_in_place(q):
    T, K, R, O = 6, 3, 10, 50
    hb = L.acts(R, O + 5, torch.bfloat16, 3).cuda()
    h = hb[:, 3:3 + O]
    pos = torch.arange(T * K, dtype=torch.int32).reshape(T, K) % R
    gates = torch.rand((T, K), generator=torch.Generator().manual_seed(1))
    yb = torch.full((T, O + 9), 4.0, dtype=torch.bfloat16, device="cuda")
    y = yb[:, 2:2 + O]
    y.copy_(L.acts(T, O, torch.bfloat16, 4))
    ref, bound = combine_ref(h, pos, gates, torch.bfloat16, y.clone())
    q.moe_combine(h, pos.cuda(), gates.cuda(), residual=y, out=y)
    L.assert_within(y, ref, bound)
    keep = yb.clone()
    keep[:, 2:2 + O] = 4.0
    assert bool((keep == 4.0).all())
    bad = pos.clone()
    bad[2, 1], bad[4, 0] = -1, R
    z = torch.isnan(q.moe_combine(h, bad.cuda(), gates.cuda())).cpu()
    assert z.all(1).tolist() == [False, False, True, False, True, False]
    assert int(z.sum()) == 2 * O


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_routed_mlp_as_used(q, T, dtype):
    """Router, group, gate/up product with SiLU gating, down product, return
    with the shared expert as residual: each step against its own reference on
    the previous step's outputs, and the plain routed experts (moe_topk) where
    it takes the token count."""
    E, K, I, F, gs = 12, 3, 256, 96, 32
    wu, su = L.int4((E, 2 * F), I, gs, 20)
    wd, sd = L.int4((E, I), F, gs, 21)
    x = L.acts(T, I, dtype, 22)
    logits = L.acts(T, E, torch.float32, 23).cuda()
    ids, gates = q.router_topk(logits, E, K)
    off, tokens, pos = q.moe_group(ids, E)
    h = q.i4g_grouped(dev(wu), dev(su), x.cuda(), off, gs, rows=tokens, act="silu", gated=True)
    d = q.i4g_grouped(dev(wd), dev(sd), h, off, gs)
    shared = q.i4g_linear(dev(wd[0]), dev(sd[0]), h[:T].contiguous(), gs)
    y = q.moe_combine(d, pos, gates, residual=shared)
    o = off.cpu().numpy()
    assert o[-1] == T * K
    tk = tokens.cpu().long()
    for e in range(E):
        lo, hi = o[e], o[e + 1]
        if hi == lo:
            continue
        ref, bound = L.reference(L.decode_int4(wu[e], su[e], I, gs), x[tk[lo:hi]], dtype,
                                 act="silu", gated=True)
        L.assert_within(h[lo:hi], ref, bound, f"up {e}")
        ref, bound = L.reference(L.decode_int4(wd[e], sd[e], F, gs), h[lo:hi], dtype)
        L.assert_within(d[lo:hi], ref, bound, f"down {e}")
    ref, bound = combine_ref(d, pos, gates, dtype, shared)
    L.assert_within(y, ref, bound)
    if T <= 8 and dtype == torch.float32:
        a = q.moe_topk(dev(wu), dev(su), ids, gates, x.cuda(), gs)
        up = q.i4g_grouped(dev(wu), dev(su), x.cuda(), off, gs, rows=tokens)
        assert L.rel_l2(q.moe_combine(up, pos, gates), a.cpu().double()) <= 1e-5


@pytest.mark.parametrize("T", [3, 60])
def test_routed_mlp_captured_and_replayed(q, T):
    """The whole chain in one graph, replayed with other routings and inputs."""
    E, K, I, F, gs = 8, 2, 256, 64, 32
    wu, su = (dev(t) for t in L.int4((E, 2 * F), I, gs, 24))
    wd, sd = (dev(t) for t in L.int4((E, I), F, gs, 25))
    x = L.acts(T, I, torch.bfloat16, 26).cuda()
    logits = L.acts(T, E, torch.float32, 27).cuda()

    def step(x, logits):
        ids, gates = q.router_topk(logits, E, K)
        off, tokens, pos = q.moe_group(ids, E)
        h = q.i4g_grouped(wu, su, x, off, gs, rows=tokens, act="silu", gated=True)
        return q.moe_combine(q.i4g_grouped(wd, sd, h, off, gs), pos, gates, residual=x)

    step(x, logits)
    xin, lin = x.clone(), logits.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(xin, lin)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(xin, lin)
    for i in range(4):
        xin.copy_(x.roll(i, 0) * (i + 1))
        lin.copy_(logits.roll(i, 1))
        g.replay()
        want = step(xin, lin)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("I,gs,gated", [(160, 32, False), (128, 64, True)])
def test_grouped_wide_tiles(q, I, gs, gated, dtype):
    """Enough rows for the wide tiles, the experts' rows filling them to every
    sixteenth."""
    counts = [1500, 7, 0, 16, 2000, 33, 100, 344, 49, 65, 81, 113]
    E, R, O = len(counts), sum(counts), 4096
    w, s = L.int4((E, O), I, gs, 40)
    off = counts_offsets(counts)
    r = np.random.default_rng(2)
    T = 600
    x = L.acts(T, I, dtype, 41)
    rows = r.integers(0, T, R).astype(np.int32)
    rows[10], rows[1507 + 3] = -1, T                 # experts 0 and 3
    y = q.i4g_grouped(dev(w), dev(s), x.cuda(), dev(off), gs, rows=dev(rows),
                      act="silu" if gated else None, gated=gated)
    bad = [10, 1507 + 3]
    assert bool(torch.isnan(y[bad]).all())
    for e in range(E):
        keep = [i for i in range(off[e], off[e + 1]) if i not in bad]
        if keep:
            ref, bound = L.reference(L.decode_int4(w[e], s[e], I, gs),
                                     x[torch.from_numpy(rows[keep]).long()], dtype,
                                     act="silu" if gated else None, gated=gated)
            L.assert_within(y[keep], ref, bound, f"expert {e}")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("counts,O", [([7, 13, 0, 16, 17, 1, 3, 20] * 8, 600),
                                      ([900, 3, 0, 400, 64, 65], 2600)])
@pytest.mark.parametrize("I,gs,gated", [(45, 2, False), (101, 64, True)])
def test_grouped_wide_general(q, counts, O, I, gs, gated, dtype):
    """Shapes of the general kernel with many tiles of 16 and of 64 rows."""
    E, R, T = len(counts), sum(counts), 50
    w, s = L.int4((E, O), I, gs, 42)
    off = counts_offsets(counts)
    x, bias = L.acts(T, I, dtype, 43), L.acts(E, O, dtype, 44)
    rows = np.random.default_rng(3).integers(0, T, R).astype(np.int32)
    k = {"act": "gelu_tanh" if gated else None, "gated": gated}
    y = q.i4g_grouped(dev(w), dev(s), x.cuda(), dev(off), gs, rows=dev(rows), bias=bias.cuda(),
                      **k)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            ref, bound = L.reference(L.decode_int4(w[e], s[e], I, gs),
                                     x[torch.from_numpy(rows[lo:hi]).long()], dtype,
                                     bias=bias[e], **k)
            L.assert_within(y[lo:hi], ref, bound, f"expert {e}")
