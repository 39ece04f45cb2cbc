"""The plan of packed sequences: every TMA map it makes on the device is byte for byte the one the encoder makes of
that sequence, whatever the sequence and the whole tensor span, and its tiles are all there, heaviest first
(plan_maps.cu; the plan runs alone, so a wrong map is compared, never read through)."""
import os
import subprocess

import pytest

from head_dim_attention_gb300 import build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_maps_and_tiles(tmp_path):
    exe = str(tmp_path / "plan_maps")
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-O1", "-o", exe, os.path.join(HERE, "plan_maps.cu"),
                    os.path.join(build.CSRC, "varlen.cu")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
