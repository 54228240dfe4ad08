"""The arithmetic of groups cut into parts (csrc/parts.hpp) near 2^31 slots, on the host, with signed overflow an
error."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_parts_near_the_most_slots(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path / "parts")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                    f"-I{os.path.join(ROOT, 'tensor_product_convolution_amd', 'csrc')}",
                    os.path.join(ROOT, "tests", "host", "parts_driver.cpp"), "-o", exe], check=True, capture_output=True, timeout=120)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
