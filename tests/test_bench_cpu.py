"""The bench's accounting, and what its reference arm loads."""
import os
import subprocess
import sys

import pytest

import bench
import quantized_linear_attention_damp_b200 as D

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("fmt", ["mixed", "int8", "fp8", "fp32"])
@pytest.mark.parametrize("name", sorted(bench.W.WORKLOADS))
def test_unit_bytes_are_the_layouts(name, fmt):
    w = bench.W.WORKLOADS[name]
    block, _ = D.damp_layout(D.FORMATS[fmt], w.d, w.d, w.hp if fmt == "mixed" else 0)
    elt = 2 if w.in_dtype == "bf16" else 4
    alpha = 4 * w.d if w.gate == bench.W.GATE_KDA else 4
    assert bench.unit_bytes(w, fmt) == 2 * block + 3 * w.d * elt + alpha + 4 + 4 * w.d


def test_the_reference_arm_loads_nothing_of_the_library():
    code = ("import runpy, sys; sys.argv = ['bench.py', '--impl', 'reference', '--steps', '1', '--workload', "
            "'tiny_gdn']; runpy.run_path('bench.py', run_name='__main__'); "
            "assert 'quantized_linear_attention_damp_b200' not in sys.modules; "
            "assert 'libdamp' not in open('/proc/self/maps').read()")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
