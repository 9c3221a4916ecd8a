"""The FP8 product's size query on the host, for sizes that the product takes
and for those that it refuses."""
import subprocess
import sys

import pytest


@pytest.fixture(scope="module")
def iqp():
    import fp4_quantized_prep_amd as m
    return m


def test_workspace_size_of_products_that_are_refused(iqp):
    """No workspace, and no end of the process (in a process of its own: a
    division by zero would be the end of it)."""
    sizes = [(1 << 38, 1 << 38, 7168), (1 << 31, 128, 7168), (128, 1 << 31, 7168), (128, 256, 257 * 128), (128, 256, 7169),
             (-128, 256, 7168), (128, -256, 7168), (128, 256, -7168), (128, 256, 0), ((1 << 63) - 1, (1 << 63) - 1, (1 << 63) - 1)]
    code = f"import fp4_quantized_prep_amd as m; print([m.fp8_gemm_workspace_bytes(*x) for x in {sizes}])"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split("\n")[0] == str([0] * len(sizes)), (r.returncode, r.stdout, r.stderr)


def test_workspace_size_of_products_that_are_taken(iqp):
    need = iqp.fp8_gemm_workspace_bytes(128, 256, 7168)
    assert need > 0 and iqp.fp8_gemm_workspace_bytes(65, 64, 256 * 128) == need
    assert iqp.fp8_gemm_workspace_bytes(2147483647, 2147483647, 7168) == 0
