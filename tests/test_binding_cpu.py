"""The package and its build where the Python binding of the attention layer's
operators is missing or does not compile."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "fp4_quantized_prep_amd")


@pytest.mark.parametrize("binding", [None, b"not a library"])
def test_package_without_the_binding(tmp_path, binding):
    """Every entry point that needs the C library alone is there; the layer's
    operators say what is missing when they are called."""
    copy = tmp_path / "fp4_quantized_prep_amd"
    copy.mkdir()
    for f in ("__init__.py", "layer.py", "libiqprep.so"):
        shutil.copy(os.path.join(PKG, f), copy / f)
    if binding is not None:
        (copy / "_binding.so").write_bytes(binding)
    code = """
import torch, fp4_quantized_prep_amd as m
assert m.library_path().startswith(%r), m.library_path()
print(m.abi_version(), m.indexer_q_workspace_bytes(16) > 0, m.fp8_gemm_workspace_bytes(128, 256, 7168) > 0)
t = torch.zeros(2, 128, dtype=torch.uint8)
c = m.fp8_kv_cache(4, 2, head_dim=64, block_size=16, device="cpu")
x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
for call in (lambda: m.fp8_gemm_1x128_128x128(t, t, t, t), lambda: m.qk_norm_rope(x, x, x, x, t, t),
             lambda: m.kv_cache_append_fp8(x, x, c, t, t, t), lambda: m.kv_cache_read_fp8(c, t, t, t, 1),
             lambda: m.attention_fp8_kv(x, c, t, t, t)):
    try:
        call()
    except ImportError as e:
        assert "_binding.so" in str(e) and "build.py" in str(e)
    else:
        raise AssertionError("no error")
print("ok")
""" % str(tmp_path)
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split("\n")[:2] == ["3 True True", "ok"], (r.stdout, r.stderr)


@pytest.mark.parametrize("fails", [None, "g++", "hipcc -shared", "hipcc -c"])
def test_a_failed_build_leaves_the_built_files(tmp_path, monkeypatch, fails):
    spec = importlib.util.spec_from_file_location("_iqp_build_test", os.path.join(PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "a.hip").write_text("")
    for name, value in (("PKG_DIR", ""), ("CSRC", "csrc"), ("LIB_PATH", b.LIB_NAME), ("BINDING_PATH", "_binding.so")):
        monkeypatch.setattr(b, name, str(tmp_path / value))
    for path in (b.LIB_PATH, b.BINDING_PATH):
        with open(path, "w") as f:
            f.write("old")

    def run(cmd, **kwargs):
        """Writes what the compiler would, or fails as it would."""
        step = "g++" if cmd[0] == "g++" else "hipcc -c" if "-c" in cmd else "hipcc -shared"
        if step == fails:
            return subprocess.CompletedProcess(cmd, 1, "", "no")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(b.subprocess, "run", run)
    if fails:
        with pytest.raises(RuntimeError):
            b.build()
    else:
        assert b.build() == b.LIB_PATH
    assert [open(p).read() for p in (b.LIB_PATH, b.BINDING_PATH)] == ["old" if fails else "new"] * 2
