"""Operands that share memory, without a GPU: the host rule against brute force
over bytes, and the entry points' refusals (fake pointers, never used)."""
import ctypes as C
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 40                 # never mapped
OVERLAP = 10


@pytest.fixture(scope="module")
def q():
    import quantized_weight_decode_amd as q
    try:
        q.lib()
    except ImportError as e:
        pytest.skip(str(e))
    return q


def test_rule_against_brute_force(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    exe = str(tmp_path / "host_rows")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I",
                    os.path.join(ROOT, "quantized_weight_decode_amd", "csrc"),
                    os.path.join(ROOT, "tests", "host_rows.cpp"), "-o", exe], check=True)
    rng = random.Random(1)
    sets, lines = [], []
    for _ in range(20000):
        two = []
        for _ in range(2):
            width = rng.randint(1, 7)
            two.append([1000 + rng.randint(0, 60), rng.randint(1, 6), width,
                        width + rng.randint(0, 12)])
        if rng.random() < 0.5:          # columns of one buffer
            ld = max(two[0][3], two[1][3])
            two[0][3] = two[1][3] = ld
        sets.append(two)
        lines.append(" ".join(str(v) for r in two for v in r))
    out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True,
                         check=True).stdout.split()
    assert len(out) == len(sets)
    shared = 0
    for two, got in zip(sets, out):
        a, b = ({p + i * ld + k for i in range(n) for k in range(w)} for p, n, w, ld in two)
        assert int(got) == bool(a & b), two
        shared += bool(a & b)
    assert 0.2 < shared / len(sets) < 0.9


def linear(q, **k):
    # 4 rows: x 4 x 64, y 4 x 8, w 8 x 32 bytes, scales 8 x 2, bias 8 in f32
    a = dict(w=A, s=A + 4096, x=A + 8192, ldx=64, y=A + 16384, ldy=8, S=4, epi=None,
             ws=A + (1 << 20))
    a.update(k)
    epi = C.addressof(a["epi"]) if a["epi"] is not None else None
    return q.qgemv_i4g_linear(a["w"], a["s"], a["x"], a["ldx"], a["y"], a["ldy"], a["S"], 64, 8,
                              32, 0, epi, a["ws"], 1 << 30, 0)


def test_product_refuses_shared_operands(q):
    E = q.Epilogue
    y = A + 16384
    assert linear(q, x=y) == OVERLAP
    assert linear(q, x=y - 4 * 64 * 4 + 4) == OVERLAP           # the last float of x
    assert linear(q, x=y + 4 * 8 * 4 - 4) == OVERLAP            # the first
    assert linear(q, w=y - 252) == OVERLAP
    assert linear(q, s=y - 60) == OVERLAP
    assert linear(q, epi=E(0, 0, y + 16, None, 0)) == OVERLAP
    assert linear(q, epi=E(0, 0, None, y + 4, 8)) == OVERLAP    # shifted by one element
    assert linear(q, epi=E(0, 0, None, y, 9)) == OVERLAP        # other stride
    assert linear(q, x=A + 8192, ldx=72, y=A + 8192 + 63 * 4, ldy=72) == OVERLAP
    assert linear(q, ws=y - (y % 256)) == OVERLAP
    assert linear(q, ws=A + 8192) == OVERLAP and linear(q, ws=A) == OVERLAP
    assert linear(q, ws=A + 32768, epi=E(0, 0, None, A + 32768, 8)) == OVERLAP


def test_grouped_refuses_shared_operands(q):
    def f(**k):
        a = dict(w=A, s=A + 4096, off=A + 8192, rows=A + 12288, x=A + 16384, y=A + 32768)
        a.update(k)
        return q.qgemv_i4g_grouped(a["w"], a["s"], 256, 16, 4, a["off"], a["rows"], a["x"], 64,
                                   4, a["y"], 8, 9, 64, 8, 32, 0, None, A + (1 << 20), 1 << 30,
                                   0)
    y = A + 32768
    for k in ("w", "s", "off", "rows", "x"):
        assert f(**{k: y}) == OVERLAP, k
    assert f(w=y - 1023) == OVERLAP and f(off=y - 16) == OVERLAP


def test_routing_refuses_shared_operands(q):
    g = q.qgemv_moe_group
    assert g(A, 2, 2, 4, A + 256, A + 512, A, None, 0, 0) == OVERLAP         # ids in place
    assert g(A, 2, 2, 4, A + 256, A + 272, A + 512, None, 0, 0) == OVERLAP   # offsets, tokens
    assert g(A, 2, 2, 4, A + 256, A + 512, A + 516, None, 0, 0) == OVERLAP   # tokens, pos
    need = q.qgemv_moe_group_workspace(4096, 8, 64)
    assert g(A, 4096, 8, 64, A + (1 << 20), A + (2 << 20), A + (3 << 20), A + (2 << 20), need,
             0) == OVERLAP
    c = q.qgemv_moe_combine
    h, pos, gates, y = A, A + 4096, A + 8192, A + 16384
    assert c(y, 8, 4, pos, gates, 2, 2, 8, None, 0, y, 8, 0, 0) == OVERLAP
    assert c(h, 8, 4, y, gates, 2, 2, 8, None, 0, y, 8, 0, 0) == OVERLAP
    assert c(h, 8, 4, pos, y + 60, 2, 2, 8, None, 0, y, 8, 0, 0) == OVERLAP
    assert c(h, 8, 4, pos, gates, 2, 2, 8, y, 9, y, 8, 0, 0) == OVERLAP
    assert c(h, 8, 4, pos, gates, 2, 2, 8, y + 4, 8, y, 8, 0, 0) == OVERLAP


def test_overlap_has_a_name(q):
    assert "overlap" in q.strerror(OVERLAP)
