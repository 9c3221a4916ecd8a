"""The FP8 product's size queries on the host, for sizes that the product takes
and for those that it refuses, and sizes for each of its kernels."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


#: Sizes, off every tile, that the product's rule sends to each of its kernels.
KERNEL_SIZES = [
    ("stream 16x16", 1, 515, 128), ("stream 16x16", 13, 2115, 1536),
    ("stream 32x16", 1, 6145, 256), ("stream 32x16", 11, 6150, 3712),
    ("stream 16x32", 17, 515, 384), ("stream 16x32", 31, 4097, 1536),
    ("stream 32x32", 17, 6145, 640), ("stream 32x32", 32, 7169, 2048),
    ("stream 16x64", 33, 515, 384), ("stream 16x64", 63, 4097, 1536),
    ("stream 32x64", 33, 6145, 256), ("stream 32x64", 61, 6150, 1536),
    ("split 64x64", 70, 515, 4096), ("split 64x64", 101, 200, 7168),
    ("tile 64x64", 70, 515, 128), ("tile 64x64", 200, 2115, 1536),
    ("tile 128x64", 130, 12300, 128), ("tile 128x64", 777, 2115, 7168),
    ("tile 128x128", 130, 12300, 1024), ("tile 128x128", 500, 6150, 2048),
    ("tile 128x128, two stages", 513, 7169, 128), ("tile 128x128, two stages", 643, 6001, 1024),
    ("tile 256x256", 1290, 6145, 128), ("tile 256x256", 1098, 7169, 640), ("tile 256x256", 4632, 8190, 1536),
]


@pytest.mark.parametrize("kernel,M,N,K", KERNEL_SIZES)
def test_kernel_of_a_size(iqp, kernel, M, N, K):
    assert iqp.debug_fp8_gemm_kernel(M, N, K) == kernel


def test_every_kernel_has_its_sizes(iqp):
    """Each kernel that the library names, and each that a grid of sizes takes."""
    with open(os.path.join(ROOT, "fp4_quantized_prep_amd", "csrc", "fp8_gemm.hip")) as f:
        named = set(re.findall(r"case GEMM_\w+: return \"([^\"]+)\";", f.read()))
    listed = {k for k, *_ in KERNEL_SIZES}
    assert listed == named and len(named) == 12
    m = sorted({round(1.37 ** i) for i in range(30)})
    taken = {iqp.debug_fp8_gemm_kernel(M, N, K, w) for M in m for N in (1, 200, 900, 2115, 4000, 6144, 9000, 20000)
             for K in (128, 512, 1536, 4096, 7168, 32768) for w in (False, True)}
    assert taken == named


def test_kernel_of_products_that_are_refused(iqp):
    assert [iqp.debug_fp8_gemm_kernel(*x) for x in ((0, 1, 128), (1, 0, 128), (1, 1, 0), (1, 1, 100), (1 << 31, 1, 128),
                                                     (1, 1, 257 * 128))] == [""] * 6
    assert iqp.debug_fp8_gemm_kernel(70, 515, 4096, workspace=False) == "tile 64x64"
