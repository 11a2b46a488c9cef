"""Refusals of the products with an epilogue and the routed slots, without a
GPU: by name, before any pointer is used."""
import ctypes as C

import pytest
import torch

BAD = 0xDEADBEEF00  # 256-byte aligned, never mapped
OK, NULL, DIMS, GS, ALIGN, IDS, WS, ARG = 0, 1, 2, 3, 4, 6, 7, 9
BIG = 1 << 40


@pytest.fixture(scope="module")
def q():
    import quantized_weight_decode_amd as q
    try:
        q.lib()
    except ImportError as e:
        pytest.skip(str(e))
    return q


def linear(q, fp8=False, **k):
    a = dict(w=BAD, s=BAD, x=BAD, ldx=64, y=BAD, ldy=8, S=3, I=64, O=8, gs=32, dtype=0, epi=None,
             ws=BAD, n=BIG)
    a.update(k)
    epi = C.addressof(a["epi"]) if a["epi"] is not None else None
    head = (a["w"], a["s"], a["x"], a["ldx"], a["y"], a["ldy"], a["S"], a["I"], a["O"])
    tail = (a["dtype"], epi, a["ws"], a["n"], 0)
    return q.qgemv_fp8b128_linear(*head, *tail) if fp8 else \
        q.qgemv_i4g_linear(*head, a["gs"], *tail)


@pytest.mark.parametrize("fp8", [False, True])
def test_linear_refusals(q, fp8):
    def f(**k):
        return linear(q, fp8, **k)
    for p in ("w", "s", "x", "y"):
        assert f(**{p: 0}) == NULL
    assert f(S=-1) == DIMS and f(S=(1 << 24) + 1) == DIMS
    assert f(I=0) == DIMS and f(I=(1 << 24) + 1, ldx=1 << 25) == DIMS
    assert f(O=0) == DIMS
    assert f(S=1 << 24, O=1 << 24, ldy=1 << 24) == DIMS            # more tiles than a launch
    assert f(ldx=63) == DIMS and f(ldy=7) == DIMS
    assert f(dtype=2) == ARG and f(dtype=-1) == ARG
    assert f(s=BAD + 2) == ALIGN and f(x=BAD + 2) == ALIGN and f(y=BAD + 1, dtype=1) == ALIGN
    assert f(ws=0) == WS and f(n=0) == WS and f(ws=BAD + 128) == WS
    assert f(n=q.qgemv_linear_workspace(3, 64, 8, 0) - 1) == WS
    E = q.Epilogue
    assert f(epi=E(5, 0, None, None, 0)) == ARG and f(epi=E(-1, 0, None, None, 0)) == ARG
    assert f(epi=E(0, 2, None, None, 0)) == ARG
    assert f(epi=E(2, 1, None, None, 0), O=7) == DIMS               # gated: even O
    assert f(epi=E(0, 0, None, BAD, 7)) == DIMS                     # residual rows overlap
    assert f(epi=E(0, 0, BAD + 1, None, 0)) == ALIGN
    assert f(epi=E(0, 0, None, BAD + 2, 8)) == ALIGN
    if not fp8:
        assert f(gs=63) == GS and f(gs=0) == GS
    # no rows: nothing is launched, whatever the pointers
    assert f(S=0, w=0, x=0, y=0, ws=0) == OK
    assert f(S=0, dtype=7) == ARG


def grouped(q, **k):
    a = dict(w=BAD, s=BAD, wst=256, sst=16, E=4, off=BAD, rows=None, x=BAD, ldx=64, T=9, y=BAD,
             ldy=8, R=9, I=64, O=8, gs=32, dtype=1, epi=None, ws=BAD, n=BIG)
    a.update(k)
    epi = C.addressof(a["epi"]) if a["epi"] is not None else None
    return q.qgemv_i4g_grouped(a["w"], a["s"], a["wst"], a["sst"], a["E"], a["off"], a["rows"],
                               a["x"], a["ldx"], a["T"], a["y"], a["ldy"], a["R"], a["I"], a["O"],
                               a["gs"], a["dtype"], epi, a["ws"], a["n"], 0)


def test_grouped_refusals(q):
    def f(**k):
        return grouped(q, **k)
    for p in ("w", "s", "off", "x", "y"):
        assert f(**{p: 0}) == NULL
    assert f(E=0) == DIMS and f(E=1025) == DIMS and f(R=-1) == DIMS
    assert f(T=8) == DIMS                                           # x[r] for 9 rows
    assert f(T=0, rows=BAD) == DIMS
    assert f(wst=255) == IDS and f(sst=15) == IDS
    assert f(off=BAD + 2) == ALIGN and f(rows=BAD + 1) == ALIGN
    assert f(gs=31) == GS and f(dtype=3) == ARG
    assert f(epi=q.Epilogue(0, 0, None, BAD, 8)) == ARG             # takes no residual
    need = q.qgemv_grouped_workspace(9, 9, 4, 64, 8, 1)
    assert need > 0 and f(n=need - 1) == WS and f(ws=BAD + 64) == WS
    assert f(R=0, T=0, w=0, x=0, y=0, off=0, ws=0) == OK


def test_group_and_combine_refusals(q):
    g = q.qgemv_moe_group
    assert g(0, 2, 2, 4, BAD, BAD, BAD, BAD, BIG, 0) == NULL
    assert g(BAD, 2, 2, 4, 0, BAD, BAD, BAD, BIG, 0) == NULL
    assert g(0, 0, 2, 4, 0, 0, 0, 0, 0, 0) == NULL                  # offsets, also for no token
    assert g(BAD, -1, 2, 4, BAD, BAD, BAD, BAD, BIG, 0) == DIMS
    assert g(BAD, 2, 0, 4, BAD, BAD, BAD, BAD, BIG, 0) == DIMS
    assert g(BAD, 2, 2, 1025, BAD, BAD, BAD, BAD, BIG, 0) == DIMS
    assert g(BAD, 1 << 23, 3, 4, BAD, BAD, BAD, BAD, BIG, 0) == DIMS
    assert g(BAD + 2, 2, 2, 4, BAD, BAD, BAD, BAD, BIG, 0) == ALIGN
    need = q.qgemv_moe_group_workspace(4096, 8, 64)
    assert need > 0
    assert g(BAD, 4096, 8, 64, BAD, BAD, BAD, BAD, need - 1, 0) == WS
    assert g(BAD, 4096, 8, 64, BAD, BAD, BAD, 0, BIG, 0) == WS
    c = q.qgemv_moe_combine
    assert c(0, 8, 4, BAD, BAD, 2, 2, 8, None, 0, BAD, 8, 0, 0) == NULL
    assert c(BAD, 8, 4, BAD, 0, 2, 2, 8, None, 0, BAD, 8, 0, 0) == NULL
    assert c(BAD, 7, 4, BAD, BAD, 2, 2, 8, None, 0, BAD, 8, 0, 0) == DIMS
    assert c(BAD, 8, 4, BAD, BAD, 2, 2, 8, BAD, 7, BAD, 8, 0, 0) == DIMS
    assert c(BAD, 8, 4, BAD, BAD, 2, 65, 8, None, 0, BAD, 8, 0, 0) == DIMS
    assert c(BAD, 8, 4, BAD, BAD, 2, 2, 8, None, 0, BAD, 8, 5, 0) == ARG
    assert c(BAD + 2, 8, 4, BAD, BAD, 2, 2, 8, None, 0, BAD, 8, 0, 0) == ALIGN
    assert c(0, 8, 0, 0, 0, 0, 2, 8, None, 0, 0, 8, 0, 0) == OK     # no tokens


def test_workspaces_of_refused_sizes_are_zero(q):
    assert q.qgemv_linear_workspace(-1, 64, 8, 0) == 0
    assert q.qgemv_linear_workspace(4, 64, 8, 9) == 0
    assert q.qgemv_grouped_workspace(4, 4, 0, 64, 8, 0) == 0
    assert q.qgemv_moe_group_workspace(4, 0, 8) == 0


def test_tensor_layer_checks_before_the_call(q):
    w, s = torch.zeros((8, 32), dtype=torch.uint8), torch.zeros((8, 2))
    x = torch.zeros((3, 64))
    with pytest.raises(TypeError, match="CUDA"):
        q.i4g_linear(w, s, x, 32)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        q.i4g_linear(w, s, x.half(), 32)
    with pytest.raises(ValueError, match="shape"):
        q.i4g_linear(w[:, :31], s, x, 32)
    with pytest.raises(q.QgemvError):
        q.i4g_linear(w, s, x, 31)
    with pytest.raises(ValueError):
        q.fp8b128_linear(torch.zeros((8, 64), dtype=torch.uint8), torch.zeros((2, 1)), x)
    with pytest.raises(ValueError, match="act"):
        q._epilogue(torch.float32, 8, None, "tanh", False, None, 3)
    with pytest.raises(ValueError, match="even"):
        q._epilogue(torch.float32, 7, None, None, True, None, 3)
    with pytest.raises(ValueError):
        q.i4g_grouped(w[None], s[None], x, torch.zeros(3, dtype=torch.int32), 32)
    with pytest.raises(ValueError):
        q.moe_group(torch.zeros(4, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        q.moe_combine(x, torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 3)))
