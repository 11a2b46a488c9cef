"""The plan of an 8-bit product, from its sizes, without a GPU (not a test module)."""
import collections
import functools
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SQUARE = 4                      # tiles: 256, 192, 128 and 64 rows x 256, and 128 x 128

Plan = collections.namedtuple("Plan", "tile kind parts head head_kind bm")


@functools.lru_cache(maxsize=None)
def _driver():
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    exe = os.path.join(tempfile.mkdtemp(prefix="matmul_plan_"), "plan")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror",
                    "-I", os.path.join(ROOT, "quantized_weight_decode_amd", "csrc"),
                    os.path.join(ROOT, "tests", "host_matmul_plan.cpp"), "-o", exe], check=True)
    return exe


def plans(queries):
    """Plans of (R, E, I, O, bf16, gated, direct, fits, CUs); E = 0: dense."""
    lines = "\n".join(" ".join(str(int(v)) for v in q) for q in queries)
    r = subprocess.run([_driver()], input=lines + "\n", capture_output=True, text=True, check=True)
    out = [Plan(*(int(v) for v in s.split())) for s in r.stdout.splitlines()]
    assert len(out) == len(queries)
    return out


def plan(R, I, O, bf16=True, gated=False, E=0, direct=True, fits=True, ncu=256):
    return plans([(R, E, I, O, bf16, gated, direct, fits, ncu)])[0]


# Dense bfloat16 products with rows on 16 bytes, one at least for each way that the tile
# kernel takes them on 256 CUs: kind of tile, whether K is cut into parts, the kind of a
# first launch for whole rounds of the CUs (None: one launch), then S, I, O, gated.
REACHED = [
    (0, False, None, 202, 128, 33448, False),
    (0, False, None, 4072, 128, 2822, True),
    (1, False, None, 3374, 128, 2348, False),
    (1, False, None, 2188, 128, 3632, True),
    (2, False, None, 4112, 9424, 776, False),
    (2, False, None, 4221, 8560, 812, False),
    (2, False, None, 4164, 8688, 832, True),
    (2, False, None, 4372, 8912, 798, True),
    (3, False, None, 67, 128, 130, False),
    (3, False, None, 67, 128, 128, True),
    (4, False, None, 4207, 128, 796, False),
    (4, False, None, 4207, 144, 770, True),
    (0, True, None, 1454, 12032, 3066, False),
    (0, True, None, 201, 7168, 16564, True),
    (1, True, None, 129, 7472, 11334, False),
    (1, True, None, 469, 15360, 5560, True),
    (2, True, None, 2625, 34304, 516, False),
    (2, True, None, 2624, 34384, 560, True),
    (3, True, None, 65, 1424, 128, False),
    (3, True, None, 66, 1472, 132, True),
    (4, True, None, 17, 8528, 10756, False),
    (4, True, None, 2238, 7520, 128, True),
    (1, False, 0, 3622, 3408, 6752, False),
    (1, False, 0, 4257, 3360, 5898, True),
    (1, False, 0, 2040, 6144, 12290, False),
    (2, False, 0, 2007, 8608, 12288, True),
    (2, False, 1, 3329, 8640, 5858, False),
    (3, False, 0, 195, 400, 66098, False),
    (3, False, 1, 899, 784, 17136, True),
    (3, False, 2, 275, 2976, 33018, False),
    (4, False, 0, 3561, 800, 6702, False),
    (4, False, 0, 3474, 1024, 6896, True),
    (4, False, 0, 2048, 6144, 12288, True),
    (4, False, 1, 4142, 1872, 4692, True),
    (1, True, 3, 3251, 42080, 2474, False),
    (3, True, 3, 2, 3712, 65586, False),
    (3, True, 3, 2, 3776, 65632, True),
    (4, True, 1, 2845, 21184, 5648, False),
]
