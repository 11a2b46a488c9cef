"""Products of two 8-bit operands, dense and grouped by expert, against 64 bits."""
import numpy as np
import pytest
import torch

from gpu_util import torch_cuda
from matmul_util import (assert_within, decode_rows, decode_weights, reference, rel_l2, rows,
                         weights)

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q():
    torch_cuda()
    import quantized_weight_decode_amd as q
    q.lib()
    return q


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def randn(shape, dtype, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def strided(t, pad):
    """t as a view of rows `pad` elements longer."""
    wide = torch.empty((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def shifted(t, by):
    """t's values from `by` bytes behind an allocation's start."""
    buf = torch.empty(t.numel() + by, dtype=torch.uint8, device=t.device)
    v = buf[by:].view(t.shape)
    v.copy_(t)
    return v


def check(q, S, I, O, dtype, act=None, gated=False, bias=False, residual=False, pad=0, shift=0,
          seed=0):
    w, s = weights((), O, I, seed + 1)
    c, cs = rows(S, I, seed + 2)
    oc = O // 2 if gated else O
    b = randn((O,), dtype, seed + 3) if bias else None
    r = randn((S, oc), dtype, seed + 4) if residual else None
    ref, bound = reference(decode_weights(w, s), decode_rows(c, cs), dtype, b, act, gated, r)
    x, xs = cuda(c), cuda(cs)
    wd = cuda(w)
    if pad:
        x, xs = strided(x, pad), strided(xs, 3)
    if shift:
        wd = shifted(wd, shift)
    y = q.fp8b128_matmul(wd, cuda(s), x, xs, bias=b.cuda() if bias else None, act=act, gated=gated,
                         residual=r.cuda() if residual else None, dtype=dtype)
    assert y.dtype == dtype and y.shape == (S, oc)
    assert_within(y, ref, bound, f"{S}x{I}x{O}")
    return y, ref


SHAPES = [(1, 1, 1), (1, 128, 16), (3, 512, 256), (2, 127, 33), (5, 129, 100), (16, 200, 64),
          (17, 384, 130), (33, 1000, 70), (64, 640, 258), (65, 256, 512), (130, 1024, 300),
          (257, 2048, 512), (300, 912, 768)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,I,O", SHAPES)
def test_plain(q, S, I, O, dtype):
    y, ref = check(q, S, I, O, DT[dtype], seed=S + I)
    if dtype == "f32":
        # over a whole output the roundings of sums average: sqrt of the number of
        # terms, here below 2^6, times 2^-24, and the final rounding
        assert rel_l2(y, ref) <= 2.0 ** -18


# (S, I, O, gated) that reach each kind of tile, whole and ragged, and K in parts
LARGE = [(2040, 384, 8192, False), (2040, 272, 8190, False), (2040, 256, 8192, True),
         (2040, 400, 8180, True), (2100, 384, 8400, False), (2100, 384, 8200, True),
         (1000, 384, 8200, False), (1000, 256, 7172, False), (1000, 256, 14336, True),
         (300, 912, 2 * 392, True)]


@pytest.mark.parametrize("S,I,O,gated", LARGE)
def test_every_tile(q, S, I, O, gated):
    check(q, S, I, O, torch.bfloat16, "silu" if gated else None, gated, bias=True, residual=True,
          seed=S + O)
    check(q, S, I, O, torch.bfloat16, None, gated, pad=16, seed=S + O + 1)


@pytest.mark.parametrize("S,I,O,gated", [(2040, 2048, 12290, False), (2040, 2048, 12288, True)])
def test_two_launches(q, S, I, O, gated):
    """More tiles than one round of the CUs: the last columns by a launch of their own."""
    check(q, S, I, O, torch.bfloat16, "relu" if gated else None, gated, bias=True, residual=True,
          seed=O)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,I,O,gated", [(40, 16384, 264, False), (300, 7168, 520, False),
                                         (257, 12048, 300, True), (70, 9001, 130, False),
                                         (130, 9001, 132, True), (16, 12288, 7168, False)])
def test_parts_of_k(q, S, I, O, gated, dtype):
    """Products cut along K; the workspace is written up to its size only."""
    need = q.qgemv_matmul_workspace(S, I, O, 1 if dtype == "bf16" else 0, int(gated))
    assert need > 0 or S <= 64
    check(q, S, I, O, DT[dtype], "gelu_tanh" if gated else None, gated, bias=True, residual=True,
          seed=S)
    w, s = weights((), O, I, S + 1)
    c, cs = rows(S, I, S + 2)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    args = (cuda(w), cuda(s), cuda(c), cuda(cs))
    y = q.fp8b128_matmul(*args, gated=gated, dtype=DT[dtype], workspace=ws[:need])
    assert (ws[need:] == 0x5A).all()
    assert torch.equal(y, q.fp8b128_matmul(*args, gated=gated, dtype=DT[dtype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
def test_epilogue(q, act, gated, dtype):
    for S, I, O in ((3, 256, 64), (40, 300, 200), (150, 512, 600), (140, 384, 290)):
        check(q, S, I, O, DT[dtype], act, gated, True, True, seed=O)
    check(q, 7, 129, 2 * 37, DT[dtype], act, gated, bias=True, seed=1)
    check(q, 140, 640, 2 * 131, DT[dtype], act, gated, residual=True, seed=2)


@pytest.mark.parametrize("pad,shift", [(16, 0), (1, 0), (0, 1), (0, 4), (3, 7), (128, 16)])
@pytest.mark.parametrize("S", [4, 40, 200])
def test_strides_and_alignment(q, S, pad, shift):
    for dtype in DT.values():
        check(q, S, 384, 272, dtype, pad=pad, shift=shift, seed=pad + shift)
        check(q, S, 272, 80, dtype, "silu", True, pad=pad, shift=shift, seed=pad + shift)


def test_every_code(q):
    """All 254 finite codes of both operands against each other: each y is one
    product, exact in f32."""
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    n = len(codes)
    one = np.ones((2, 1), np.float32)
    for S in (n, 5):
        x = codes[:S, None].copy()
        y = q.fp8b128_matmul(cuda(codes[:, None].copy()), cuda(one), cuda(x),
                             torch.ones((S, 1), device="cuda"), dtype=torch.float32)
        v = torch.from_numpy(codes).view(torch.float8_e4m3fn).double()
        assert torch.equal(y.cpu().double(), v[:S, None] * v[None, :])
        # and at every place of a block, bfloat16: one product each, rounded once
        for k in (0, 7, 8, 63, 64, 100, 127):
            xk = np.zeros((S, 128), np.uint8)
            wk = np.zeros((n, 128), np.uint8)
            xk[:, k], wk[:, k] = codes[:S], codes
            y = q.fp8b128_matmul(cuda(wk), cuda(one), cuda(xk), torch.ones((S, 1), device="cuda"))
            assert torch.equal(y.cpu(), (v[:S, None] * v[None, :]).bfloat16())


@pytest.mark.parametrize("S", [3, 90, 260])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_codes_of_every_size_together(q, S, dtype):
    """Subnormal codes, zeros and the largest ones side by side, in both operands."""
    I, O = 640, 260
    w, s = weights((), O, I, 40)
    r = np.random.default_rng(41)
    c = weights((), S, I, 42)[0]
    small = (r.integers(0, 8, (S, I)) | r.integers(0, 2, (S, I)) << 7).astype(np.uint8)
    c = np.where(r.random((S, I)) < 0.5, small, c)
    w = np.where(r.random((O, I)) < 0.3, r.integers(0, 8, (O, I)).astype(np.uint8), w)
    c[:, ::128] = w[:, ::128] = 0x38                 # 1 in every block
    cs = np.exp(r.uniform(-3, 3, (S, 5))).astype(np.float32)
    ref, bound = reference(decode_weights(w, s), decode_rows(c, cs), DT[dtype])
    y = q.fp8b128_matmul(cuda(w), cuda(s), cuda(c), cuda(cs), dtype=DT[dtype])
    assert_within(y, ref, bound)
    # groups of eight where only subnormal codes meet large ones
    c[:, 8:] = 1
    w[:, 8:] = 0x7E
    w[:, 9::8] = 0x01
    c[:, ::128] = w[:, ::128] = 0x38
    ref, bound = reference(decode_weights(w, s), decode_rows(c, cs), DT[dtype])
    y = q.fp8b128_matmul(cuda(w), cuda(s), cuda(c), cuda(cs), dtype=DT[dtype])
    assert_within(y, ref, bound)


@pytest.mark.parametrize("S", [2, 60, 260])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_stays_in_its_row_and_column(q, S, dtype):
    I, O = 400, 300
    w, s = weights((), O, I, 5)
    c, cs = rows(S, I, 6)
    ref, bound = reference(decode_weights(w, s), decode_rows(c, cs), DT[dtype])
    w[37, 399] = 0xFF
    w[290, 0] = 0x7F
    c[1, 130] = 0x7F
    s2, cs2 = s.copy(), cs.copy()
    s2[1, 2] = np.nan                             # rows 128..255
    cs2[S - 1, 3] = np.nan
    y = q.fp8b128_matmul(cuda(w), cuda(s), cuda(c), cuda(cs), dtype=DT[dtype]).cpu().double()
    bad = torch.zeros(S, O, dtype=torch.bool)
    bad[:, 37] = bad[:, 290] = True
    bad[1] = True
    assert torch.equal(y.isnan(), bad)
    assert_within(torch.where(bad, ref, y), ref, bound)
    y = q.fp8b128_matmul(cuda(w), cuda(s2), cuda(c), cuda(cs2), dtype=DT[dtype]).cpu().double()
    bad[:, 128:256] = True
    bad[S - 1] = True
    assert torch.equal(y.isnan(), bad)


@pytest.mark.parametrize("S", [3, 50, 200])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scales_of_every_size(q, S, dtype):
    """Activation scales from 2^-126 (a row of zeros) to 2^100 next to each other: a
    row's result goes by its own."""
    I, O = 300, 150
    w, s = weights((), O, I, 7)
    c, cs = rows(S, I, 8)
    cs = cs * np.exp2(np.random.default_rng(9).integers(-100, 100, (S, 1))).astype(np.float32)
    c[0] = 0
    cs[0] = 2.0 ** -126
    ref, bound = reference(decode_weights(w, s), decode_rows(c, cs), DT[dtype])
    y = q.fp8b128_matmul(cuda(w), cuda(s), cuda(c), cuda(cs), dtype=DT[dtype])
    assert_within(y, ref, bound)
    assert not y[0].any()


@pytest.mark.parametrize("S", [1, 37, 200])
def test_only_its_rows_are_written(q, S):
    I, O = 256, 130
    w, s = weights((), O, I, 10)
    c, cs = rows(S, I, 11)
    ref, bound = reference(decode_weights(w, s), decode_rows(c, cs), torch.bfloat16)
    buf = torch.full((S + 2, O + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:S + 1, 4:4 + O]
    y = q.fp8b128_matmul(cuda(w), cuda(s), cuda(c), cuda(cs), out=out)
    assert y is out
    assert_within(out, ref, bound)
    out.fill_(7.0)
    assert (buf == 7.0).all()
    # the residual in place, codes as float8, and one vector
    res = randn((S, O), torch.float32, 12)
    ref, bound = reference(decode_weights(w, s), decode_rows(c, cs), torch.float32, residual=res)
    y = res.cuda()
    q.fp8b128_matmul(cuda(w).view(torch.float8_e4m3fn), cuda(s),
                     cuda(c).view(torch.float8_e4m3fn), cuda(cs), residual=y, out=y)
    assert_within(y, ref, bound)
    one = q.fp8b128_matmul(cuda(w), cuda(s), cuda(c[0]), cuda(cs[0]), residual=res[0].cuda())
    assert one.shape == (O,)
    assert_within(one[None], ref[:1], bound[:1])


def test_no_rows(q):
    w, s = weights((), 16, 128, 1)
    y = q.fp8b128_matmul(cuda(w), cuda(s), torch.empty((0, 128), dtype=torch.uint8, device="cuda"),
                         torch.empty((0, 1), device="cuda"))
    assert y.shape == (0, 16)


def routing(T, K, E, seed, empty=()):
    r = np.random.default_rng(seed)
    allowed = np.array([e for e in range(E) if e not in empty])
    return np.stack([r.choice(allowed, K, replace=False) for _ in range(T)]).astype(np.int32)


def grouped_reference(w, s, c, cs, offsets, rowix, dtype, bias, act, gated):
    W = decode_weights(w, s)
    x = decode_rows(c, cs)
    ref, bound = [], []
    for e in range(len(W)):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        ix = torch.arange(lo, hi) if rowix is None else rowix[lo:hi].long()
        v, d = reference(W[e], x[ix], dtype, bias[e] if bias is not None else None, act, gated)
        ref.append(v)
        bound.append(d)
    return torch.cat(ref), torch.cat(bound)


GROUPED = [(1, 1, 4, 128, 16), (4, 2, 8, 200, 48), (16, 4, 8, 384, 130), (70, 2, 5, 256, 270),
           (300, 2, 4, 512, 300), (33, 8, 64, 640, 64), (600, 1, 3, 272, 528),
           (1100, 1, 2, 256, 528)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,K,E,I,O", GROUPED)
def test_grouped(q, T, K, E, I, O, gather, dtype):
    ids = cuda(routing(T, K, E, T + E, empty=(1,) if E > K + 1 else ()))
    offsets, tokens, pos = q.moe_group(ids, E)
    w, s = weights((E,), O, I, 13)
    c, cs = rows(T if gather else T * K, I, 14)
    for act, gated, bias in ((None, False, False), ("silu", True, True)):
        b = randn((E, O), DT[dtype], 15) if bias else None
        ref, bound = grouped_reference(w, s, c, cs, offsets.cpu(), tokens.cpu() if gather else None,
                                       DT[dtype], b, act, gated)
        y = q.fp8b128_matmul_grouped(cuda(w), cuda(s), cuda(c), cuda(cs), offsets,
                                     rows=tokens if gather else None,
                                     bias=b.cuda() if bias else None, act=act, gated=gated,
                                     dtype=DT[dtype])
        assert_within(y, ref, bound, f"{T}x{K}x{E}x{I}x{O}")


@pytest.mark.parametrize("many", [False, True])
def test_grouped_rows_that_are_left_and_bad_indices(q, many):
    T, E, I, O = (300, 4, 256, 144) if many else (12, 4, 256, 144)
    R = T
    w, s = weights((E,), O, I, 16)
    c, cs = rows(T, I, 17)
    lo = [2, R // 3, R // 3, R // 2, R - 3]                  # expert 1 empty
    rowix = torch.from_numpy(np.random.default_rng(18).integers(0, T, R).astype(np.int32))
    good = rowix.clone()
    rowix[5] = T
    rowix[R // 2 + 1] = -1
    rowix[0] = rowix[R - 1] = 1 << 30                        # of no expert: not looked at
    rowix[1] = rowix[R - 2] = -(1 << 31)
    offsets = torch.tensor(lo, dtype=torch.int32)
    ref, bound = grouped_reference(w, s, c, cs, offsets, good.clamp(0, T - 1), torch.bfloat16, None,
                                   None, False)
    out = torch.full((R, O), 5.0, dtype=torch.bfloat16, device="cuda")
    y = q.fp8b128_matmul_grouped(cuda(w), cuda(s), cuda(c), cuda(cs), offsets.cuda(),
                                 rows=rowix.cuda(), out=out).cpu().double()
    assert (y[:2] == 5.0).all() and (y[R - 3:] == 5.0).all()
    mid = y[2:R - 3]
    bad = torch.zeros(len(mid), dtype=torch.bool)
    bad[5 - 2] = bad[R // 2 + 1 - 2] = True
    assert mid[bad].isnan().all()
    assert_within(mid[~bad], ref[~bad], bound[~bad])
    # offsets outside 0..R are clamped, decreasing ones name no rows
    out.fill_(5.0)
    wild = torch.tensor([-7, 4, 2, R + 100, 1 << 30], dtype=torch.int32)
    y = q.fp8b128_matmul_grouped(cuda(w), cuda(s), cuda(c), cuda(cs), wild.cuda(),
                                 out=out).cpu().double()
    ref, bound = grouped_reference(w[[0, 2]], s[[0, 2]], c, cs, [0, 4, 4], None, torch.bfloat16,
                                   None, None, False)
    assert_within(y[:2], ref[:2], bound[:2])
    last, lb = reference(decode_weights(w, s)[2], decode_rows(c, cs)[4:], torch.bfloat16)
    assert_within(y[4:], last, lb)


def test_two_calls_at_once_and_replays(q):
    """Dense and grouped products on two streams, then captured together and
    replayed over new inputs, against the same calls alone."""
    E, I, O, T, K = 8, 640, 272, 90, 2
    w, s = weights((E,), O, I, 19)
    wd, sd = cuda(w), cuda(s)
    sets = []
    for i in range(4):
        c, cs = rows(T, I, 20 + i)
        sets.append((cuda(c), cuda(cs), *q.moe_group(cuda(routing(T, K, E, 30 + i)), E)))

    def both(x, xs, off, tok, out=None):
        a = q.fp8b128_matmul(wd[0], sd[0], x, xs, act="silu", gated=True)
        b = q.fp8b128_matmul_grouped(wd, sd, x, xs, off, rows=tok)
        return a, b
    alone = [tuple(t.clone() for t in both(*v[:4])) for v in sets]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            r1 = both(*sets[0][:4])
        with torch.cuda.stream(s2):
            r2 = both(*sets[1][:4])
        torch.cuda.synchronize()
        for got, want in zip(r1 + r2, alone[0] + alone[1]):
            assert torch.equal(got, want)
    fixed = [t.clone() for t in sets[0][:4]]
    with torch.cuda.stream(s1):
        both(*fixed)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both(*fixed)
    for i in (1, 2, 3, 0, 2):
        for t, v in zip(fixed, sets[i]):
            t.copy_(v)
        g.replay()
        eager = both(*sets[3][:4])                           # eager work between replays
        torch.cuda.synchronize()
        for u, v in zip(got, alone[i]):
            assert torch.equal(u, v)
        for u, v in zip(eager, alone[3]):
            assert torch.equal(u, v)


def test_weights_and_rows_beyond_4_gb(q):
    """Offsets that pass 32 bits: the last rows of W, and the last rows of x through
    an index, against the same rows alone."""
    I, O = 65536, 65664                                  # 4.3 GB of codes
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    g = torch.Generator(device="cuda")
    g.manual_seed(50)
    w = torch.randint(0, 126, (O, I), dtype=torch.uint8, generator=g, device="cuda")
    s = torch.rand((O // 128, I // 128), generator=g, device="cuda") * 1e-3
    x, xs = q.fp8_quantize(torch.randn((70, I), generator=g, device="cuda"))
    last = slice(O - 256, O)
    xd = decode_rows(x, xs)
    ref, bound = reference(decode_weights(w[last].cpu().numpy(), s[-2:].cpu().numpy()), xd,
                           torch.bfloat16)
    for S in (3, 70):
        y = q.fp8b128_matmul(w, s, x[:S], xs[:S])
        assert_within(y[:, last], ref[:S], bound[:S], f"{S} rows")
    # W's rows as activations: T rows of x of 4.3 GB, read through an index
    ws = torch.rand((O, I // 128), generator=g, device="cuda")
    pick = torch.tensor([O - 1, 5, O - 3, 65535, 32768] * 8, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    wx, sx = x[:64].contiguous(), torch.rand((1, I // 128), generator=g, device="cuda") * 1e-3
    y = q.fp8b128_matmul_grouped(wx[None], sx[None], w, ws, offsets, rows=pick)
    ref, bound = reference(decode_weights(wx.cpu().numpy(), sx.cpu().numpy()),
                           decode_rows(w[pick.long()], ws[pick.long()]), torch.bfloat16)
    assert_within(y, ref, bound)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parts_on_two_streams_and_replayed(q, dtype):
    """Products cut along K, whose parts lie in a workspace: two at once, and captured,
    against the same calls alone."""
    S, I, O = 200, 7168, 520
    w, s = weights((), O, I, 60)
    wd, sd = cuda(w), cuda(s)
    assert q.qgemv_matmul_workspace(S, I, O, 1 if dtype == "bf16" else 0, 0) > 0
    sets = [tuple(cuda(t) for t in rows(S, I, 61 + i)) for i in range(3)]

    def call(x, xs):
        return q.fp8b128_matmul(wd, sd, x, xs, act="relu", dtype=DT[dtype])
    alone = [call(*v).clone() for v in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(call(*sets[i]))
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i], alone[i])
    fixed = [t.clone() for t in sets[0]]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = call(*fixed)
    for i in (1, 2, 0, 1):
        for t, v in zip(fixed, sets[i]):
            t.copy_(v)
        g.replay()
        eager = call(*sets[2])
        torch.cuda.synchronize()
        assert torch.equal(y, alone[i]) and torch.equal(eager, alone[2])
