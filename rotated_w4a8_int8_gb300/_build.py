"""Builds libconvrot.so in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel; the shared library links the
CUDA runtime dynamically so that it shares one runtime with the host process.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libconvrot.so")
# the binding's compiled module, named for this interpreter: another version does not load it
MARSHAL = os.path.join(HERE, "_marshal" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
# (source, object, defines): quant.cu is compiled twice, once without and once
# with the kernels that write code-norm bounds; gemm_fused.cu once per output type
SOURCES = [("api.cu", "api", []), ("quant.cu", "quant", []),
           ("quant.cu", "quant_norm", ["-DCONVROT_QUANT_NORM=1"]), ("gemm.cu", "gemm", []),
           ("int8_probe.cu", "int8_probe", []), ("decode_gemm_probe.cu", "decode_gemm_probe", []),
           ("norm_quant.cu", "norm_quant", []), ("rope.cu", "rope", []), ("gemm_few.cu", "gemm_few", []),
           *(("gemm_fused.cu", f"gemm_fused_{name}", [f"-DCONVROT_FUSED_OUT=CONVROT_{name.upper()}"])
             for name in ("bf16", "fp16", "fp32"))]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the ConvRot CUDA library cannot be built")
    return cand


def _compile(unit, extra: list[str]) -> str:
    src, name, defines = unit
    obj = os.path.join(BUILD, name + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *defines, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _python_include() -> str | None:
    """Where Python.h lies, or None: the library (C ABI) does not need it."""
    paths = sysconfig.get_paths()
    for name in ("include", "platinclude"):
        if os.path.exists(os.path.join(paths[name], "Python.h")):
            return paths[name]
    return None


def _compile_marshal() -> None:
    """The CPython extension that marshals the block operators' arguments."""
    include = _python_include()
    if include is None:
        sys.stderr.write("Python.h not found: libconvrot.so is built without the Python calls of rms_norm_quant, "
                         "qk_norm_rope and gemm_fused\n")
        return
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        raise RuntimeError("no C compiler found for the marshalling module")
    tmp = MARSHAL + ".tmp"
    cmd = [cc, "-O2", "-std=c11", "-shared", "-fPIC", "-I", include, os.path.join(CSRC, "marshal.c"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"marshal.c failed to compile:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)


def build(verbose_ptxas: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "convrot.h")]
    newest = max(os.path.getmtime(d) for d in deps)

    def current(f: str) -> bool:
        return not force and os.path.exists(f) and os.path.getmtime(f) > newest
    if current(LIB):
        if _python_include() and not current(MARSHAL):
            _compile_marshal()
        return LIB
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        marshal = ex.submit(_compile_marshal)
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
        marshal.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose_ptxas="-v" in sys.argv, force="-f" in sys.argv))
