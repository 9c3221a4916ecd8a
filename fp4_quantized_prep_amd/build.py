"""Builds libiqprep.so (the HIP kernels and the C ABI) for gfx950 in-tree, and
the host-only Python binding of the attention layer's calls (_binding.so).

    python fp4_quantized_prep_amd/build.py

(run as a script: importing the package itself needs the built files).

Compiles every csrc/*.hip with hipcc into fp4_quantized_prep_amd/libiqprep.so.
hipcc cross-compiles, so no GPU is needed to build.
"""
import concurrent.futures
import glob
import os
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libiqprep.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
BINDING_PATH = os.path.join(PKG_DIR, "_binding.so")
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    return "hipcc"


def compile_flags() -> list:
    return [
        f"--offload-arch={ARCH}",
        "-O3",
        "-std=c++17",
        "-fPIC",
        "-Wall",
        # packed fp32 VALU forms are kept out of every kernel
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        f"-I{INCLUDE}",
        f"-I{CSRC}",
    ]


def build(verbose: bool = False) -> str:
    """Compile and link the library and the binding; returns the library's path.
    Raises on failure, and then leaves the built files as they were."""
    sources = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    if not sources:
        raise RuntimeError(f"no HIP sources under {CSRC}")
    obj_dir = os.path.join(PKG_DIR, "_build")
    os.makedirs(obj_dir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        cmd = [hipcc()] + compile_flags() + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        return obj

    # one hipcc per source, a few at a time (each is single-threaded)
    jobs = max(1, min(8, len(os.sched_getaffinity(0))))
    with concurrent.futures.ThreadPoolExecutor(jobs) as pool:
        objs = list(pool.map(compile_one, sources))
    lib = os.path.join(obj_dir, LIB_NAME)     # under its own name, which the binding records
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", lib] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    binding = build_binding(obj_dir, verbose)
    os.replace(lib, LIB_PATH)
    os.replace(binding, BINDING_PATH)
    return LIB_PATH


def build_binding(lib_dir: str, verbose: bool = False) -> str:
    """Compile csrc/binding.cpp against torch and lib_dir's libiqprep.so, into
    lib_dir; host code only."""
    import sysconfig

    import torch
    import torch.utils.cpp_extension as ext
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    path = os.path.join(lib_dir, os.path.basename(BINDING_PATH))
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
           "-DUSE_ROCM=1", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f"-I{INCLUDE}"] + [f"-isystem{d}" for d in ext.include_paths() + ["/opt/rocm/include", sysconfig.get_paths()["include"]]]
    cmd += [os.path.join(CSRC, "binding.cpp"), "-o", path, f"-L{torch_lib}", "-lc10", "-ltorch_cpu", "-ltorch_python", "-lc10_hip",
            f"-L{lib_dir}", f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the binding's build failed:\n{res.stdout}\n{res.stderr}")
    return path


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
