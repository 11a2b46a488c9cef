"""Refusals of the 8-bit products, their quantizer and the gradients of routed
rows, without a GPU: by name, before any pointer is used."""
import ctypes as C

import pytest
import torch

A = 1 << 40                     # operands far apart, never mapped
OK, NULL, DIMS, ALIGN, IDS, WS, ARG, OVERLAP = 0, 1, 2, 4, 6, 7, 9, 10


@pytest.fixture(scope="module")
def q():
    import quantized_weight_decode_amd as q
    try:
        q.lib()
    except ImportError as e:
        pytest.skip(str(e))
    return q


def _epi(e):
    return C.addressof(e) if e is not None else None


def quantize(q, **k):
    a = dict(x=A, ldx=200, S=3, I=200, dtype=0, c=2 * A, ldc=200, s=3 * A, lds=2)
    a.update(k)
    return q.qgemv_fp8_quantize(a["x"], a["ldx"], a["S"], a["I"], a["dtype"], a["c"], a["ldc"],
                                a["s"], a["lds"], 0)


def test_quantize_refusals(q):
    def f(**k):
        return quantize(q, **k)
    for p in ("x", "c", "s"):
        assert f(**{p: 0}) == NULL
    assert f(S=-1) == DIMS and f(S=(1 << 24) + 1) == DIMS and f(I=0) == DIMS
    assert f(I=(1 << 24) + 1, ldx=1 << 25, ldc=1 << 25, lds=1 << 20) == DIMS
    assert f(ldx=199) == DIMS and f(ldc=199) == DIMS and f(lds=1) == DIMS
    assert f(dtype=2) == ARG
    assert f(x=A + 2) == ALIGN and f(x=A + 1, dtype=1) == ALIGN and f(s=3 * A + 2) == ALIGN
    assert f(c=A + 64) == OVERLAP and f(s=A + 64) == OVERLAP and f(s=2 * A + 64) == OVERLAP
    assert f(S=0, x=0, c=0, s=0) == OK


def matmul(q, **k):
    a = dict(w=A, ws=2 * A, x=3 * A, ldx=200, xs=4 * A, lds=2, y=5 * A, ldy=8, S=3, I=200, O=8,
             dtype=0, epi=None, wsp=7 * A, n=1 << 30)
    a.update(k)
    return q.qgemv_fp8b128_matmul(a["w"], a["ws"], a["x"], a["ldx"], a["xs"], a["lds"], a["y"],
                                  a["ldy"], a["S"], a["I"], a["O"], a["dtype"], _epi(a["epi"]),
                                  a["wsp"], a["n"], 0)


def test_matmul_refusals(q):
    def f(**k):
        return matmul(q, **k)
    E = q.Epilogue
    for p in ("w", "ws", "x", "xs", "y"):
        assert f(**{p: 0}) == NULL
    assert f(S=-1) == DIMS and f(S=(1 << 24) + 1) == DIMS and f(I=0) == DIMS and f(O=0) == DIMS
    assert f(S=1 << 24, O=1 << 24, ldy=1 << 24) == DIMS
    assert f(ldx=199) == DIMS and f(ldy=7) == DIMS and f(lds=1) == DIMS
    assert f(dtype=2) == ARG and f(dtype=-1) == ARG
    assert f(ws=2 * A + 2) == ALIGN and f(xs=4 * A + 2) == ALIGN and f(y=5 * A + 2) == ALIGN
    assert f(epi=E(5, 0, None, None, 0)) == ARG and f(epi=E(0, 2, None, None, 0)) == ARG
    assert f(epi=E(2, 1, None, None, 0), O=7) == DIMS
    assert f(epi=E(0, 0, None, 6 * A, 7)) == DIMS
    assert f(epi=E(0, 0, 6 * A + 1, None, 0)) == ALIGN
    for p in ("w", "ws", "x", "xs"):
        assert f(**{p: 5 * A + 16 - (16 if p in ("ws", "xs") else 3)}) == OVERLAP
    assert f(epi=E(0, 0, 5 * A + 8, None, 0)) == OVERLAP
    assert f(epi=E(0, 0, None, 5 * A + 8, 8)) == OVERLAP
    assert f(S=0, w=0, ws=0, x=0, xs=0, y=0, wsp=0) == OK
    assert f(S=0, dtype=7) == ARG
    # sizes that are cut along K need a workspace
    big = dict(S=300, I=7168, ldx=7168, lds=56, O=7168, ldy=7168, dtype=1)
    need = q.qgemv_matmul_workspace(300, 7168, 7168, 1, 0)
    assert need > 0
    assert f(wsp=0, **big) == WS and f(wsp=7 * A + 128, **big) == WS and f(n=need - 1, **big) == WS
    assert f(wsp=5 * A, **big) == OVERLAP and f(wsp=A, **big) == OVERLAP
    assert q.qgemv_matmul_workspace(0, 64, 64, 0, 0) == 0
    assert q.qgemv_matmul_workspace(3, 64, 63, 0, 1) == 0


def grouped(q, **k):
    a = dict(w=A, ws=2 * A, wst=1600, sst=2, E=4, off=6 * A, rows=None, x=3 * A, ldx=200, xs=4 * A,
             lds=2, T=9, y=5 * A, ldy=8, R=9, I=200, O=8, dtype=1, epi=None, wsp=7 * A, n=1 << 20)
    a.update(k)
    return q.qgemv_fp8b128_matmul_grouped(a["w"], a["ws"], a["wst"], a["sst"], a["E"], a["off"],
                                          a["rows"], a["x"], a["ldx"], a["xs"], a["lds"], a["T"],
                                          a["y"], a["ldy"], a["R"], a["I"], a["O"], a["dtype"],
                                          _epi(a["epi"]), a["wsp"], a["n"], 0)


def test_grouped_refusals(q):
    def f(**k):
        return grouped(q, **k)
    E = q.Epilogue
    for p in ("w", "ws", "x", "xs", "off", "y"):
        assert f(**{p: 0}) == NULL
    assert f(E=0) == DIMS and f(E=1025) == DIMS and f(R=-1) == DIMS and f(T=-1) == DIMS
    assert f(T=8) == DIMS and f(T=0, rows=8 * A) == DIMS
    assert f(ldx=199) == DIMS and f(ldy=7) == DIMS and f(lds=1) == DIMS
    assert f(wst=1599) == IDS and f(sst=1) == IDS
    assert f(off=6 * A + 2) == ALIGN and f(rows=8 * A + 1) == ALIGN and f(xs=4 * A + 2) == ALIGN
    assert f(dtype=3) == ARG and f(epi=E(0, 0, None, 8 * A, 8)) == ARG       # residual
    assert f(wsp=0) == WS and f(wsp=7 * A + 128) == WS
    assert f(n=q.qgemv_matmul_grouped_workspace(9, 4) - 1) == WS
    assert f(wsp=5 * A) == OVERLAP and f(wsp=6 * A) == OVERLAP and f(wsp=4 * A) == OVERLAP
    assert f(rows=5 * A + 4) == OVERLAP and f(xs=5 * A) == OVERLAP
    assert f(R=0, T=0, w=0, ws=0, x=0, xs=0, off=0, y=0, wsp=0) == OK


@pytest.mark.parametrize("E,R", [(1024, 1 << 15), (1, 1 << 15)])
def test_grouped_sizes_beyond_a_launch(q, E, R):
    O, B = 1 << 24, 1 << 58
    st = grouped(q, E=E, R=R, T=R, O=O, ldy=O, wst=O * 200, sst=1 << 18, w=0x1000, ws=B, x=2 * B,
                 xs=3 * B, y=4 * B, off=5 * B, wsp=6 * B, n=1 << 40)
    assert st == DIMS


def test_routed_refusals(q):
    def d(x=A, ldx=8, T=4, t=2 * A, R=6, I=8, y=3 * A, ldy=8, dtype=0):
        return q.qgemv_moe_dispatch(x, ldx, T, t, R, I, y, ldy, dtype, 0)
    assert d(x=0) == NULL and d(t=0) == NULL and d(y=0) == NULL
    assert d(T=-1) == DIMS and d(R=-1) == DIMS and d(I=0) == DIMS and d(R=(1 << 24) + 1) == DIMS
    assert d(ldx=7) == DIMS and d(ldy=7) == DIMS and d(dtype=2) == ARG
    assert d(x=A + 2) == ALIGN and d(t=2 * A + 1) == ALIGN and d(y=3 * A + 1, dtype=1) == ALIGN
    assert d(y=A + 32) == OVERLAP and d(y=2 * A + 4) == OVERLAP
    assert d(R=0, x=0, t=0, y=0) == OK

    def g(dy=A, lddy=8, R=6, p=2 * A, T=4, K=2, I=8, dx=3 * A, lddx=8, dtype=0):
        return q.qgemv_moe_dispatch_grad(dy, lddy, R, p, T, K, I, dx, lddx, dtype, 0)
    assert g(dy=0) == NULL and g(p=0) == NULL and g(dx=0) == NULL
    assert g(K=0) == DIMS and g(K=65) == DIMS and g(T=-1) == DIMS and g(I=0) == DIMS
    assert g(lddy=7) == DIMS and g(lddx=7) == DIMS and g(dtype=-1) == ARG
    assert g(dy=A + 2) == ALIGN and g(p=2 * A + 2) == ALIGN and g(dx=3 * A + 1, dtype=1) == ALIGN
    assert g(dx=A + 32) == OVERLAP and g(dx=2 * A) == OVERLAP
    assert g(T=0, dy=0, p=0, dx=0) == OK

    def c(dy=A, lddy=8, h=2 * A, ldh=8, R=6, t=3 * A, p=4 * A, g=5 * A, T=3, K=2, O=8, dh=6 * A,
          lddh=8, dg=7 * A, dtype=0):
        return q.qgemv_moe_combine_grad(dy, lddy, h, ldh, R, t, p, g, T, K, O, dh, lddh, dg, dtype,
                                        0)
    for k in ("dy", "h", "t", "p", "g", "dh", "dg"):
        assert c(**{k: 0}) == NULL
        if k not in ("dh", "dg"):
            assert c(**{k: 6 * A + 16}) == OVERLAP and c(**{k: 7 * A}) == OVERLAP
    assert c(dg=6 * A + 4) == OVERLAP
    assert c(K=0) == DIMS and c(K=65) == DIMS and c(T=-1) == DIMS and c(O=0) == DIMS
    assert c(lddy=7) == DIMS and c(ldh=7) == DIMS and c(lddh=7) == DIMS and c(dtype=2) == ARG
    assert c(dy=A + 2) == ALIGN and c(h=2 * A + 1, dtype=1) == ALIGN and c(dg=7 * A + 2) == ALIGN
    assert c(t=3 * A + 2) == ALIGN and c(p=4 * A + 1) == ALIGN and c(g=5 * A + 2) == ALIGN
    assert c(T=0, dy=0, h=0, t=0, p=0, g=0, dh=0, dg=0) == OK


def meta(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_tensor_layer(q):
    """Sizes that a C int would wrap, gradients, shapes and types, with tensors that
    are never read."""
    f32, i32, BIG = {"dtype": torch.float32}, {"dtype": torch.int32}, (1 << 32) + 3
    w, s, x, xs = meta(8, 200), meta(1, 2, **f32), meta(3, 200), meta(3, 2, **f32)

    def refused(f, *a, **k):
        with pytest.raises(q.QgemvError) as e:
            f(*a, **k)
        assert e.value.status == DIMS
    refused(q.fp8_quantize, meta(BIG, 200, **f32))
    refused(q.fp8b128_matmul, w, s, meta(BIG, 200), meta(BIG, 2, **f32))
    refused(q.fp8b128_matmul_grouped, meta(2, 8, 200), meta(2, 1, 2, **f32), x, xs,
            meta(3, **i32), rows=meta(BIG, **i32))
    refused(q.moe_dispatch, meta(4, 8, **f32), meta(BIG, **i32))
    refused(q.moe_dispatch_grad, meta(BIG, 8, **f32), meta(4, 2, **i32))
    refused(q.moe_combine_grad, meta(4, BIG, **f32), meta(8, BIG, **f32), meta(8, **i32),
            meta(4, 2, **i32), meta(4, 2, **f32))

    def asks(t):
        return t.clone().requires_grad_()
    h, pos, gates, tok = meta(8, 8, **f32), meta(4, 2, **i32), meta(4, 2, **f32), meta(8, **i32)
    dy = meta(4, 8, **f32)
    calls = [lambda g: q.fp8_quantize(g(meta(3, 200, **f32))),
             lambda g: q.fp8b128_matmul(w, s, x, g(xs)),
             lambda g: q.fp8b128_matmul(w, g(s), x, xs),
             lambda g: q.fp8b128_matmul(w, s, x, xs, bias=g(meta(8, **f32))),
             lambda g: q.fp8b128_matmul(w, s, x, xs, residual=g(meta(3, 8, **f32))),
             lambda g: q.fp8b128_matmul_grouped(meta(2, 8, 200), meta(2, 1, 2, **f32), x, g(xs),
                                                meta(3, **i32)),
             lambda g: q.moe_dispatch(g(dy), tok), lambda g: q.moe_dispatch_grad(g(h), pos),
             lambda g: q.moe_combine_grad(g(dy), h, tok, pos, gates),
             lambda g: q.moe_combine_grad(dy, g(h), tok, pos, gates),
             lambda g: q.moe_combine_grad(dy, h, tok, pos, g(gates))]
    for f in calls:
        with pytest.raises(ValueError, match="gradient"):
            f(asks)
        with torch.no_grad(), pytest.raises(TypeError, match="CUDA"):
            f(asks)
        with pytest.raises(TypeError, match="CUDA"):
            f(lambda t: t)
    with pytest.raises(ValueError, match="scale_inv"):
        q.fp8b128_matmul(w, meta(1, 1, **f32), x, xs)
    with pytest.raises(ValueError, match="w must have shape"):
        q.fp8b128_matmul(meta(8, 199), s, x, xs)
    with pytest.raises(TypeError, match="dtype"):
        q.fp8b128_matmul(w, s, x, xs, dtype=torch.float16)
    with pytest.raises(TypeError, match="x must be"):
        q.fp8_quantize(meta(3, 200, dtype=torch.float16))
    with pytest.raises(ValueError, match="tokens"):
        q.moe_combine_grad(dy, h, meta(7, **i32), pos, gates)
