"""Vectors of eight f32 elements are loaded and stored as 16-byte aligned: the calls
check their operands' rows for 16 bytes, not for 32."""
import os
import re
import subprocess

import pytest

import quantized_weight_decode_amd.build as build


def test_eight_floats_promise_16_bytes(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("needs hipcc")
    out = str(tmp_path / "quantize.ll")
    flags = [f for f in build.HIPFLAGS if f not in ("-shared", "-Wall")]
    src = os.path.join(build.CSRC, "quantize.hip")
    r = subprocess.run([build.HIPCC, *flags, "--cuda-device-only", "-S", "-emit-llvm", src, "-o",
                        out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    with open(out) as f:
        loads = re.findall(r"<8 x float>.*align (\d+)", f.read())
    assert loads and all(int(a) <= 16 for a in loads), loads
