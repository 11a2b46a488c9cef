"""Products with an epilogue (i4g_linear, fp8b128_linear) on the GPU against
64-bit references, elementwise within the bound derived in linear_util."""
import numpy as np
import pytest
import torch

import linear_util as L
from gpu_util import dev, torch_cuda

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.bfloat16]
# (S, I, O, gs): one row to several tiles, both sides of 16, 32, 64 and 128
# rows; odd and tiny I and O; group sizes in and out of whole 32 columns
SHAPES = [(1, 512, 256, 64), (1, 1, 1, 2), (2, 6144, 130, 64), (3, 64, 7, 32), (5, 3, 18, 2),
          (15, 160, 66, 32), (16, 4096, 48, 128), (17, 33, 65, 2), (31, 96, 129, 96),
          (33, 2048, 258, 64), (64, 416, 514, 32), (65, 100, 64, 48), (96, 1024, 300, 64),
          (128, 640, 255, 128), (130, 1001, 257, 100), (257, 1536, 1026, 64),
          (300, 2080, 70, 256), (520, 256, 1000, 64)]


@pytest.fixture(scope="module")
def q():
    torch_cuda()
    import quantized_weight_decode_amd as q
    return q


def _run(q, fmt, S, I, O, gs, dtype, seed=0, **k):
    if fmt == "i4g":
        w, s = L.int4((O,), I, gs, seed)
        W = L.decode_int4(w, s, I, gs)
    else:
        w, s = L.fp8(O, I, seed)
        W = L.decode_fp8(w, s)
    x = L.acts(S, I, dtype, seed + 1)
    gated = k.get("gated", False)
    oc = O // 2 if gated else O
    bias = L.acts(1, O, dtype, seed + 2)[0] if k.get("bias") else None
    res = L.acts(S, oc, dtype, seed + 3) if k.get("residual") else None
    kw = {"act": k.get("act"), "gated": gated}
    dv = {"bias": bias.cuda() if bias is not None else None,
          "residual": res.cuda() if res is not None else None}
    if fmt == "i4g":
        y = q.i4g_linear(dev(w), dev(s), x.cuda(), gs, **kw, **dv)
    else:
        y = q.fp8b128_linear(dev(w), dev(s), x.cuda(), **kw, **dv)
    ref, bound = L.reference(W, x, dtype, bias=bias, residual=res, **kw)
    return y, ref, bound


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("S,I,O,gs", SHAPES)
def test_i4g_product(q, S, I, O, gs, dtype):
    y, ref, bound = _run(q, "i4g", S, I, O, gs, dtype, seed=S + I)
    L.assert_within(y, ref, bound)
    if dtype == torch.float32:
        assert L.rel_l2(y, ref) <= 1e-5


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("S,I,O", [(s, i, o) for s, i, o, _ in SHAPES])
def test_fp8_product(q, S, I, O, dtype):
    y, ref, bound = _run(q, "fp8", S, I, O, 128, dtype, seed=S + I)
    L.assert_within(y, ref, bound)
    if dtype == torch.float32:
        assert L.rel_l2(y, ref) <= 1e-5


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("fmt", ["i4g", "fp8"])
@pytest.mark.parametrize("S,I,O,gs", [(1, 512, 250, 64), (7, 129, 34, 2), (40, 768, 132, 32),
                                      (140, 512, 516, 64)])
@pytest.mark.parametrize("act,gated,bias,residual",
                         [("relu", False, True, False), ("silu", False, False, True),
                          ("gelu", False, True, True), ("gelu_tanh", False, False, False),
                          (None, False, True, True), ("silu", True, False, False),
                          ("gelu", True, True, True), (None, True, False, True),
                          ("gelu_tanh", True, True, False), ("relu", True, False, False)])
def test_epilogue(q, fmt, S, I, O, gs, act, gated, bias, residual, dtype):
    y, ref, bound = _run(q, fmt, S, I, O, gs, dtype, act=act, gated=gated, bias=bias,
                         residual=residual)
    L.assert_within(y, ref, bound)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("S", [1, 6, 50, 200])
def test_strided_rows_and_untouched_gaps(q, S, dtype):
    """x, residual and out as column slices of wider tensors; the columns
    beside out and the rows behind it keep their values; odd offsets leave the
    rows on element alignment only."""
    I, O, gs = 320, 90, 64
    w, s = L.int4((O,), I, gs, 3)
    xb = L.acts(S + 2, I + 37, dtype, 4).cuda()
    rb = L.acts(S + 2, O + 11, dtype, 5).cuda()
    ob = torch.full((S + 2, O + 23), 7.5, dtype=dtype, device="cuda")
    x, r, out = xb[1:S + 1, 5:5 + I], rb[1:S + 1, 3:3 + O], ob[1:S + 1, 7:7 + O]
    y = q.i4g_linear(dev(w), dev(s), x, gs, residual=r, out=out)
    assert y.data_ptr() == out.data_ptr()
    ref, bound = L.reference(L.decode_int4(w, s, I, gs), x, dtype, residual=r)
    L.assert_within(out, ref, bound)
    keep = ob.clone()
    keep[1:S + 1, 7:7 + O] = 7.5
    assert bool((keep == 7.5).all())


@pytest.mark.parametrize("S", [1, 20, 150])
def test_residual_in_place_and_vector_form(q, S):
    I, O, gs = 256, 192, 64
    w, s = L.int4((O,), I, gs, 6)
    x = L.acts(S, I, torch.bfloat16, 7)
    h = L.acts(S, O, torch.bfloat16, 8)
    y = h.cuda()
    q.i4g_linear(dev(w), dev(s), x.cuda(), gs, residual=y, out=y)
    ref, bound = L.reference(L.decode_int4(w, s, I, gs), x, torch.bfloat16, residual=h)
    L.assert_within(y, ref, bound)
    v = q.i4g_linear(dev(w), dev(s), x[0].cuda(), gs, residual=h[0].cuda())
    assert v.shape == (O,)
    L.assert_within(v[None], ref[:1], bound[:1])


@pytest.mark.parametrize("fmt", ["i4g", "fp8"])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("S", [4, 40, 140])
def test_wide_range_and_non_finite_rows(q, fmt, S, dtype):
    """Rows of very different scale, an outlier on one column, a row of zeros;
    a row with an infinity or NaN comes out without finite sums and leaves the
    others alone."""
    I, O, gs = 512, 130, 64
    w, s = L.int4((O,), I, gs, 9) if fmt == "i4g" else L.fp8(O, I, 9)
    W = L.decode_int4(w, s, I, gs) if fmt == "i4g" else L.decode_fp8(w, s)
    x = L.acts(S, I, dtype, 10)
    x[0] *= 1e-30
    x[1] *= 1e25
    x[2, 77] = 3e4
    x[3] = 0.0
    call = (lambda v: q.i4g_linear(dev(w), dev(s), v.cuda(), gs)) if fmt == "i4g" else \
        (lambda v: q.fp8b128_linear(dev(w), dev(s), v.cuda()))
    ref, bound = L.reference(W, x, dtype)
    L.assert_within(call(x), ref, bound)
    bad = x.clone()
    bad[1, 5], bad[2, 500] = float("nan"), float("inf")
    y = call(bad)
    assert not bool(torch.isfinite(y[1]).any()) and not bool(torch.isfinite(y[2]).any())
    rest = [i for i in range(S) if i not in (1, 2)]
    L.assert_within(y[rest], ref[rest], bound[rest])


@pytest.mark.parametrize("S", [2, 100])
def test_nan_weight_code_poisons_its_column_only(q, S):
    I, O = 256, 140
    w, s = L.fp8(O, I, 11)
    w[77, 33] = 0x7F
    x = L.acts(S, I, torch.bfloat16, 12)
    y = q.fp8b128_linear(dev(w), dev(s), x.cuda())
    assert bool(torch.isnan(y[:, 77]).all())
    assert bool(torch.isfinite(y[:, [c for c in range(O) if c != 77]]).all())


def test_single_and_many_rows_agree_with_the_gemv(q):
    """The plain f32 product next to the library's GEMV of the same weights."""
    I, O, gs = 2048, 512, 64
    w, s = L.int4((O,), I, gs, 13)
    x = L.acts(4, I, torch.float32, 14).cuda()
    a = q.i4g_linear(dev(w), dev(s), x, gs)
    b = q.i4g(dev(w), dev(s), x, gs)
    assert L.rel_l2(a, b.cpu().double()) <= 1e-5


@pytest.mark.parametrize("S", [0, 1, 3, 70, 300])
def test_results_do_not_change_between_calls(q, S):
    I, O, gs = 1024, 400, 64
    w, s = (dev(t) for t in L.int4((O,), I, gs, 15))
    x = L.acts(S, I, torch.bfloat16, 16).cuda()
    y = [q.i4g_linear(w, s, x, gs, act="silu", gated=True) for _ in range(3)]
    assert y[0].shape == (S, O // 2)
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


@pytest.mark.parametrize("S", [1, 40, 200])
def test_side_stream_and_replayed_graphs(q, S):
    """Work goes to the current stream; two captured calls with a workspace
    each replay several times, with eager calls and new inputs between."""
    I, O, gs = 768, 300, 64
    w, s = (dev(t) for t in L.int4((O,), I, gs, 17))
    x = L.acts(S, I, torch.bfloat16, 18).cuda()
    want = q.i4g_linear(w, s, x, gs, act="silu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = q.i4g_linear(w, s, x, gs, act="silu")
    side.synchronize()
    assert torch.equal(got, want)
    graphs = []
    for _ in range(2):
        xin, out = x.clone(), torch.zeros_like(want)
        ws = q.linear_workspace(S, I, O, x.dtype, "cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.i4g_linear(w, s, xin, gs, act="silu", workspace=ws, out=out)
        graphs.append((g, xin, out))
    for i in range(4):
        for j, (g, xin, out) in enumerate(graphs):
            xin.copy_(x * (1 + i + 2 * j))
            out.zero_()
            g.replay()
        want = [q.i4g_linear(w, s, xin, gs, act="silu") for _, xin, _ in graphs]
        torch.cuda.synchronize()
        for (_, _, out), v in zip(graphs, want):
            assert torch.equal(out, v)


@pytest.mark.parametrize("S", [3, 140])
def test_rows_beyond_32_bit_offsets(q, S):
    """y rows 2^30 bytes apart or so: the last row starts past 4 GiB."""
    I, O, gs = 64, 40, 32
    w, s = L.int4((O,), I, gs, 19)
    x = L.acts(S, I, torch.bfloat16, 20)
    ld = (5 << 30) // 2 // (S - 1)
    buf = torch.empty((S - 1) * ld + I, dtype=torch.bfloat16, device="cuda")
    out = buf.as_strided((S, O), (ld, 1))
    q.i4g_linear(dev(w), dev(s), x.cuda(), gs, out=out)
    ref, bound = L.reference(L.decode_int4(w, s, I, gs), x, torch.bfloat16)
    L.assert_within(out, ref, bound)
    xs = buf.as_strided((S, I), (ld, 1))
    xs.copy_(x)
    y = q.i4g_linear(dev(w), dev(s), xs, gs)
    L.assert_within(y, ref, bound)


def test_misaligned_weights(q):
    """w one byte off any alignment: the general kernel's result."""
    I, O, gs = 256, 60, 64
    w, s = L.int4((O,), I, gs, 21)
    buf = torch.zeros(w.size + 64, dtype=torch.uint8, device="cuda")
    for off in (1, 4, 8):
        v = buf[off:off + w.size].view(O, I // 2)
        v.copy_(dev(w))
        for S in (2, 90):
            x = L.acts(S, I, torch.bfloat16, 22)
            ref, bound = L.reference(L.decode_int4(w, s, I, gs), x, torch.bfloat16)
            L.assert_within(q.i4g_linear(v, dev(s), x.cuda(), gs), ref, bound)




# products large enough for the wide tiles: 128, 96 and 64 rows (bf16), 64 and
# 32 rows (f32); half K steps (I % 64 == 32), scale groups of 32, 64 and 96
@pytest.mark.parametrize("fmt", ["i4g", "fp8"])
@pytest.mark.parametrize("S,O,dtype", [(2000, 4000, torch.bfloat16), (2060, 4100, torch.bfloat16),
                                       (900, 4000, torch.bfloat16), (1000, 4000, torch.float32),
                                       (500, 4000, torch.float32)])
@pytest.mark.parametrize("I,gs,gated", [(160, 32, False), (256, 64, True), (96, 96, False),
                                        (32, 32, True), (448, 64, False)])
def test_wide_tiles(q, fmt, S, O, dtype, I, gs, gated):
    k = {"act": "silu", "gated": True, "bias": True, "residual": True} if gated else {}
    y, ref, bound = _run(q, fmt, S, I, O, gs, dtype, seed=S + I, **k)
    L.assert_within(y, ref, bound)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("outlier", [1e4, 1e6])
@pytest.mark.parametrize("S", [2, 20, 60, 200])
def test_outlier_on_a_zero_weight_column(q, S, outlier, dtype):
    """A column whose weights are all zero takes a large activation: its size
    must not cost the other columns their bits (f32: relative L2 1e-5)."""
    I, O, gs = 2048, 256, 64
    w, s = L.int4((O,), I, gs, 30)
    w[:, 100] = 0x88                                 # q = 8, columns 200 and 201
    W = L.decode_int4(w, s, I, gs)
    x = L.acts(S, I, dtype, 31)
    x[:, 200] = outlier
    y = q.i4g_linear(dev(w), dev(s), x.cuda(), gs)
    ref, bound = L.reference(W, x, dtype)
    if dtype == torch.float32:
        assert L.rel_l2(y, ref) <= 1e-5
    else:
        # bf16's rounding and the outlier's share of the offset form: two
        # roundings of 24 |x| s per scale group
        extra = 2 * L.U * 48 * outlier * 0.02
        L.assert_within(y, ref, bound + extra)


def test_more_activations_than_one_slice(q):
    """Rows whose packed form exceeds 4 GB run in slices: rows on both sides of
    the cut against the same rows alone."""
    I, O, S, gs = 1 << 20, 64, 2100, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w = torch.randint(0, 256, (O, I // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = 0.002 + 0.018 * torch.rand((O, I // gs), device="cuda", generator=g)
    x = torch.randn((S, I), dtype=torch.bfloat16, device="cuda", generator=g)
    r = torch.randn((S, O), dtype=torch.bfloat16, device="cuda", generator=g)
    y = q.i4g_linear(w, s, x, gs, residual=r)
    for lo in (0, 1900, 2070):
        part = q.i4g_linear(w, s, x[lo:lo + 30], gs, residual=r[lo:lo + 30])
        # the same exact products in other orders: 2^20 of rms 5 * 0.012 in f32
        # sums, one bf16 rounding each
        d = (part.double() - y[lo:lo + 30].double()).abs()
        assert float((d / (2.0 ** -7 * y[lo:lo + 30].double().abs() + 0.05)).max()) <= 1.0


@pytest.mark.parametrize("fmt", ["i4g", "fp8"])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("S,O", [(100, 3700), (900, 2000), (5, 26000)])
@pytest.mark.parametrize("I,gs,gated", [(45, 2, False), (70, 6, True), (101, 64, True),
                                        (161, 10, False)])
def test_wide_general(q, fmt, S, O, dtype, I, gs, gated):
    """Shapes of the general kernel with many tiles of 16 and of 64 rows."""
    k = {"act": "gelu", "gated": True, "bias": True, "residual": True} if gated else {}
    y, ref, bound = _run(q, fmt, S, I, O, gs, dtype, seed=S + I, **k)
    L.assert_within(y, ref, bound)


def test_two_streams_at_once(q):
    """Calls of all kernels on two streams side by side, a workspace each."""
    gs, cases = 64, []
    for S, I, O in [(3, 2048, 1000), (40, 2048, 1000), (300, 1024, 4000), (60, 1001, 900)]:
        w, s = L.int4((O,), I, gs, S)
        cases.append((dev(w), dev(s), L.acts(S, I, torch.bfloat16, S + 1).cuda()))
    want = [q.i4g_linear(w, s, x, gs, act="silu") for w, s, x in cases]
    wsp = [[q.linear_workspace(x.shape[0], x.shape[1], w.shape[0], x.dtype, "cuda")
            for w, s, x in cases] for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for j, st in enumerate(streams):
            order = range(len(cases)) if j else reversed(range(len(cases)))
            with torch.cuda.stream(st):
                for c in order:
                    w, s, x = cases[c]
                    got[j].append((c, q.i4g_linear(w, s, x, gs, act="silu", workspace=wsp[j][c])))
    torch.cuda.synchronize()
    for c, y in got[0] + got[1]:
        assert torch.equal(y, want[c])


# more workgroups of 16 rows x 64 rows of W than CUs: the stream kernel with 32
# rows, and the narrow kernel
NARROW = [(20, 9000), (40, 6100), (100, 2500), (300, 1002),
          (20, 17000), (40, 8300), (100, 4200), (300, 1702)]


@pytest.mark.parametrize("fmt", ["i4g", "fp8"])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("S,O", NARROW)
@pytest.mark.parametrize("I,gs,gated", [(160, 32, False), (256, 64, True), (96, 96, False),
                                        (544, 32, True), (1024, 128, False), (32, 32, False)])
def test_narrow_tiles(q, fmt, S, O, dtype, I, gs, gated):
    k = {"act": "silu", "gated": True, "bias": True, "residual": True} if gated else {}
    y, ref, bound = _run(q, fmt, S, I, O, gs, dtype, seed=S + I, **k)
    L.assert_within(y, ref, bound)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("S,O", NARROW)
def test_narrow_tiles_rows_apart(q, S, O, dtype):
    """Strided x, residual and out, gaps untouched; rows of very different scale,
    an outlier, a row of zeros, a row with an infinity and one with NaN."""
    I, gs = 320, 64
    w, s = L.int4((O,), I, gs, 50)
    x = L.acts(S, I, dtype, 51)
    x[0] *= 1e-30
    x[1] *= 1e25
    x[2, 77] = 3e4
    x[3] = 0.0
    res = L.acts(S, O, dtype, 52)
    ref, bound = L.reference(L.decode_int4(w, s, I, gs), x, dtype, residual=res)
    x[4, 5], x[5, 300] = float("nan"), float("inf")
    xb = torch.zeros((S + 2, I + 37), dtype=dtype, device="cuda")
    rb = torch.zeros((S + 2, O + 11), dtype=dtype, device="cuda")
    ob = torch.full((S + 2, O + 23), 7.5, dtype=dtype, device="cuda")
    xs, rs, out = xb[1:S + 1, 5:5 + I], rb[1:S + 1, 3:3 + O], ob[1:S + 1, 7:7 + O]
    xs.copy_(x)
    rs.copy_(res)
    y = q.i4g_linear(dev(w), dev(s), xs, gs, residual=rs, out=out)
    assert not bool(torch.isfinite(y[4:6]).any())
    keep = [i for i in range(S) if i not in (4, 5)]
    L.assert_within(y[keep], ref[keep], bound[keep])
    ob[1:S + 1, 7:7 + O] = 7.5
    assert bool((ob == 7.5).all())


@pytest.mark.parametrize("outlier", [1e4, 1e6])
@pytest.mark.parametrize("S,O", NARROW)
def test_narrow_tiles_outlier_on_a_zero_weight_column(q, S, O, outlier):
    I, gs = 1024, 64
    w, s = L.int4((O,), I, gs, 53)
    w[:, 100] = 0x88
    x = L.acts(S, I, torch.float32, 54)
    x[:, 200] = outlier
    ref, _ = L.reference(L.decode_int4(w, s, I, gs), x, torch.float32)
    assert L.rel_l2(q.i4g_linear(dev(w), dev(s), x.cuda(), gs), ref) <= 1e-5


@pytest.mark.parametrize("S,O", NARROW)
def test_narrow_tiles_replayed_graph(q, S, O):
    I, gs = 512, 64
    w, s = (dev(t) for t in L.int4((O,), I, gs, 55))
    x = L.acts(S, I, torch.bfloat16, 56).cuda()
    q.i4g_linear(w, s, x, gs, act="silu")
    xin, ws = x.clone(), q.linear_workspace(S, I, O, x.dtype, "cuda")
    out = torch.zeros((S, O), dtype=x.dtype, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.i4g_linear(w, s, xin, gs, act="silu", workspace=ws, out=out)
    for i in range(4):
        xin.copy_(x * (1 + i))
        out.zero_()
        g.replay()
        want = q.i4g_linear(w, s, xin, gs, act="silu")
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_more_packed_activations_than_one_slice(q):
    """test_more_activations_than_one_slice with columns enough for the tiles."""
    I, O, S, gs = 1 << 20, 160, 2100, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    w = torch.randint(0, 256, (O, I // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = 0.002 + 0.018 * torch.rand((O, I // gs), device="cuda", generator=g)
    x = torch.randn((S, I), dtype=torch.bfloat16, device="cuda", generator=g)
    y = q.i4g_linear(w, s, x, gs)
    for lo in (0, 1900, 2070):
        part = q.i4g_linear(w, s, x[lo:lo + 30], gs)
        d = (part.double() - y[lo:lo + 30].double()).abs()
        assert float((d / (2.0 ** -7 * y[lo:lo + 30].double().abs() + 0.05)).max()) <= 1.0
