"""Build libtq2.so (HIP, gfx950) in the package directory with hipcc.

Usage: ``python -m gemv_tq2_g128_amd.build`` or ``build()`` from Python.
"""

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG_DIR), "include")
LIB_NAME = "libtq2.so"
SOURCES = ["tq2_api.hip", "tq2_reformat.hip", "tq2_gemv.hip", "tq2_gemm.hip", "tq2_q4.hip",
           "tq2_kv_append.hip", "tq2_attn.hip", "tq2_attn_tile.hip",
           "tq2_layer_api.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # Code object v5: loadable by the HIP runtime PyTorch ships as well.
    "-mcode-object-version=5",
    "-shared",
    # No packed-FP32 instructions anywhere in the device code.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc_path():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    p = os.path.join(rocm, "bin", "hipcc")
    return p if os.path.exists(p) else "hipcc"


PROBE_LIB_NAME = "libtq2_probe.so"
PROBE_SOURCES = ["tq2_probe.hip"]
BINDING_NAME = "_binding.so"
BINDING_SOURCE = "tq2_binding.cpp"


def build(verbose: bool = False) -> str:
    """Compile every HIP source into ``libtq2.so`` (and the benchmark's
    reference kernels into ``libtq2_probe.so``); returns the library path.
    Where PyTorch is installed, the tensor marshalling of ``attn`` and ``q4``
    is compiled into ``_binding.so`` as well; the C ABI does without it."""
    _compile(PROBE_SOURCES, PROBE_LIB_NAME, verbose)
    lib = _compile(SOURCES, LIB_NAME, verbose)
    if importlib.util.find_spec("torch") is not None:
        _compile_binding(verbose)
    else:
        print("PyTorch is not installed: %s is left out" % BINDING_NAME, flush=True)
    return lib


def host_compiler():
    """g++, or the clang++ that hipcc itself comes with."""
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return shutil.which("g++") or os.path.join(rocm, "llvm", "bin", "clang++")


def _compile_binding(verbose):
    """The host-only Python module, against PyTorch's headers and libtq2.so."""
    import torch
    root = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    out = os.path.join(PKG_DIR, BINDING_NAME)
    tmp = out + ".tmp%d" % os.getpid()
    includes = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(rocm, "include"), sysconfig.get_paths()["include"]]
    _run([host_compiler(), "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
          "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
          *("-I" + i for i in includes), os.path.join(CSRC, BINDING_SOURCE), "-o", tmp,
          "-L" + PKG_DIR, "-l:" + LIB_NAME, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu",
          "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN"], verbose)
    os.replace(tmp, out)


def _run(cmd, verbose):
    """Run one compiler command; its output, or RuntimeError."""
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # hipcc's host pass does not know the device-only target feature; drop that noise.
    noise = "is not a recognized feature for this target"
    msg = "\n".join(l for l in res.stdout.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError("%s failed (%d):\n%s" % (os.path.basename(cmd[0]), res.returncode, msg))
    if verbose and msg.strip():
        print(msg)


def _compile(sources, lib_name, verbose):
    """One object per source, in parallel, then the link."""
    out = os.path.join(PKG_DIR, lib_name)
    tmp = out + ".tmp%d" % os.getpid()
    flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory(prefix="tq2_build_") as work:
        objs = [os.path.join(work, s + ".o") for s in sources]
        cmds = [[hipcc_path(), *flags, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, s),
                 "-o", o] for s, o in zip(sources, objs)]
        with ThreadPoolExecutor(max_workers=min(len(cmds), 8)) as pool:
            list(pool.map(lambda c: _run(c, verbose), cmds))
        try:
            _run([hipcc_path(), *HIPCC_FLAGS, "-Wl,-soname," + lib_name, *objs, "-o", tmp], verbose)
        except RuntimeError:
            if os.path.exists(tmp):
                os.remove(tmp)
            raise
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
