"""Build libmoew2.so (all HIP sources under csrc/) for gfx950 with hipcc, and _bind (csrc/bind.cpp, the
compiled part of the Python binding, host code, an extension module of this Python and this PyTorch) with
g++, in-tree. The library needs hipcc alone: it is linked whatever becomes of the binding, which is left
out where PyTorch is not installed."""
import concurrent.futures
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoew2.so")
BIND = os.path.join(HERE, "_bind" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILD_DIR = os.path.join(HERE, "_build")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # packed-FP32 VALU forms are kept out of every device code object
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-result",
]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src):
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [HIPCC] + FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
    if r.returncode:
        raise RuntimeError(f"hipcc failed for {src}:\n{out}")
    return obj, out


def _build_bind():
    import torch
    from torch.utils import cpp_extension
    tmp = BIND + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DMOEW2_TORCH_VERSION="{torch.__version__}"']
    for d in cpp_extension.include_paths() + [sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", d]
    cmd += [os.path.join(CSRC, "bind.cpp"), "-o", tmp, "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        raise RuntimeError("g++ failed for bind.cpp:\n" + r.stdout + r.stderr)
    os.replace(tmp, BIND)
    return r.stdout + r.stderr


def _link(objs):
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)


def build(verbose=False):
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        bind = ex.submit(_build_bind) if importlib.util.find_spec("torch") else None
        results = list(ex.map(_compile, srcs))
        _link([o for o, _ in results])
        outs = [out for _, out in results] + ([bind.result()] if bind else ["PyTorch is not installed: no Python binding"])
    if verbose:
        for out in outs:
            if out.strip():
                print(out)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
