"""The argument validation of the layer's operators, and of experts' and adapters',
under host ASan and UBSan (CPU only): sanitize_abi's library and child process,
with the tests of these modules that take only the library."""
import glob
import os

import pytest

MODULES = ("test_layer_abi_cpu", "test_moe_abi_cpu", "test_moe_sizes_cpu")


def test_validation_clean_under_asan_ubsan(monkeypatch, capfd):
    sanitize_abi = pytest.importorskip("sanitize_abi")     # (not where GPU tests alone are run)
    if not glob.glob(os.path.join(sanitize_abi.PKG_DIR, "_build", "*.o")):
        pytest.skip("the library's objects are not built here (run the build first)")
    if not glob.glob("/opt/rocm/lib/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"):
        pytest.skip("no host ASan runtime in this image")
    one = "import test_abi_cpu as T\n"
    assert one in sanitize_abi.CHILD
    # one module after the other, each from its own namespace
    joined = "import types\nT = types.SimpleNamespace()\nfor m in %r:\n    for k, v in vars(__import__(m)).items():\n" \
             "        setattr(T, k if not hasattr(T, k) else k + '_' + m, v)\n" % (MODULES,)
    monkeypatch.setattr(sanitize_abi, "CHILD", sanitize_abi.CHILD.replace(one, joined))
    rc = sanitize_abi.main()
    out, err = capfd.readouterr()
    assert rc == 0, out + err[-3000:]
    assert int(out.split()[0]) >= 15 and "argument-check tests passed under ASan/UBSan" in out
