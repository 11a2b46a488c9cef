"""The library holds the tile kernels that a plan can name, and no others."""
import re
import shutil
import subprocess

import pytest

from matmul_plan_util import SQUARE, plan


@pytest.fixture(scope="module")
def kernels():
    """(type, fragments of W and of x, rows on 16 bytes, grouped) of the built kernels."""
    import quantized_weight_decode_amd as q
    try:
        q.lib()
    except ImportError as e:
        pytest.skip(str(e))
    if shutil.which("nm") is None:
        pytest.skip("needs nm")
    names = subprocess.run(["nm", "-C", q.LIB_PATH], capture_output=True, text=True, check=True)
    found = set()
    for m in re.findall(r"matmul_tile<qg::(\w+), ([^>]*)>", names.stdout):
        wf, tf, _, _, _, _, _, direct, grouped = m[1].split(", ")
        found.add((m[0], int(wf), int(tf), direct == "true", grouped == "true"))
    assert found
    return found


def test_grouped_kernels(kernels):
    # kinds of tiles by their fragments: 256, 192, 128 and 64 rows, 128 x 128
    kinds = [(8, 4), (8, 3), (8, 2), (8, 1), (4, 4)]
    named = set()
    for bf16 in (False, True):
        for direct in (False, True):
            for R in (17, 300, 1 << 13, 1 << 20):
                p = plan(R, 1024, 1024, bf16=bf16, direct=direct, E=8)
                assert p.tile
                named.add(("BF16" if bf16 else "F32", *kinds[p.kind], direct, True))
    assert {k for k in kernels if k[4]} == named


def test_dense_kernels(kernels):
    want = {("BF16", 8, n, True, False) for n in (1, 2, 3, 4)}
    want |= {(t, 4, 4, d, False) for t in ("F32", "BF16") for d in (False, True)}
    assert {k for k in kernels if not k[4]} == want
    assert plan(300, 1024, 768, bf16=False).kind == SQUARE
