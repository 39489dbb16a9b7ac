"""Build the CUDA library ``_lib/libckv.so`` for sm_103a and the tensor binding
``_lib/ckv_binding.so`` over it (in-tree, no cmake).

Translation units are compiled in parallel with nvcc / g++ and linked with
``nvcc -shared``.  Only one ``-gencode`` target is emitted: GB300 (sm_103a).
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libckv.so")
BINDING = os.path.join(LIBDIR, "ckv_binding.so")
BINDING_OF = os.path.join(LIBDIR, "ckv_binding.txt")  # the torch that it was built for

GENCODE = "-gencode=arch=compute_103a,code=sm_103a"
CUDA_SOURCES = ["kpool.cu", "c128.cu", "prefill_tma.cu", "planner_device.cu", "validate.cu", "probe.cu",
                "step_maps.cu", "norm_rope.cu", "fp4_rows.cu", "fp4_attention.cu",
                "fp4_attention_rows.cu", "kv_append.cu", "kv_attention.cu", "kv_attention_few.cu",
                "tree_masks.cu",
                "merge_attention.cu", "capi.cu"]
CXX_SOURCES = ["planner.cpp"]
BINDING_SOURCE = "binding.cpp"  # CPython module over torch tensors, linked against the library


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libckv")


def _headers():
    return [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh"))] + [os.path.join(INCLUDE, "ckv.h")]


def _newer(made, sources) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(s) <= os.path.getmtime(made) for s in sources)


def _library_up_to_date() -> bool:
    return _newer(LIB, [os.path.join(CSRC, s) for s in CUDA_SOURCES + CXX_SOURCES] + _headers())


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    return spec.submodule_search_locations[0]


def _torch_build() -> str:
    """The torch and the interpreter that the module's C++ interface belongs to."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"python {sys.version}\n{_torch_dir()}\n{f.read()}"


def _binding_up_to_date() -> bool:
    try:
        with open(BINDING_OF) as f:
            built_for = f.read()
        now = _torch_build()
    except (OSError, RuntimeError):
        return False
    return built_for == now and _newer(BINDING, [os.path.join(CSRC, BINDING_SOURCE), os.path.join(INCLUDE, "ckv.h")])


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


def _compile(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _link(made, cmd):
    tmp = made + f".tmp{os.getpid()}"
    _compile([*cmd[:1], "-o", tmp, *cmd[1:]])
    os.replace(tmp, made)


def _binding_object() -> str:
    """Compile the tensor binding; needs the headers of torch and of Python."""
    obj = os.path.join(BUILD, BINDING_SOURCE + ".o")
    inc = os.path.join(_torch_dir(), "include")
    _compile(["g++", "-O2", "-std=c++17", "-fPIC", f"-I{INCLUDE}", f"-I{inc}",
              f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
              f"-I{sysconfig.get_paths()['include']}", "-I/usr/local/cuda/include", "-c",
              os.path.join(CSRC, BINDING_SOURCE), "-o", obj])
    return obj


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    """Build what is out of date.  The C library needs neither torch nor Python headers, so a tensor
    binding that cannot be built (the serving-step calls then raise) is a warning here."""
    library, binding = force or not _library_up_to_date(), force or not _binding_up_to_date()
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    cmds, objs = [], []
    if library:
        nvcc = _nvcc()
        common = ["-O3", "-std=c++17", f"-I{INCLUDE}", f"-I{CSRC}"]
        for s in CUDA_SOURCES:
            o = os.path.join(BUILD, s + ".o")
            cmd = [nvcc, GENCODE, "-lineinfo", *common, "-Xcompiler", "-fPIC", "-c",
                   os.path.join(CSRC, s), "-o", o]
            if verbose_ptxas:
                cmd.insert(1, "-Xptxas=-v")
            cmds.append(cmd)
            objs.append(o)
        for s in CXX_SOURCES:
            o = os.path.join(BUILD, s + ".o")
            cmds.append(["g++", "-O2", "-std=c++17", "-fPIC", f"-I{INCLUDE}", f"-I{CSRC}",
                         "-I/usr/local/cuda/include", "-c", os.path.join(CSRC, s), "-o", o])
            objs.append(o)
    with cf.ThreadPoolExecutor(max_workers=jobs or len(cmds) + 1) as ex:
        bind = ex.submit(_binding_object) if binding else None
        logs = list(ex.map(_compile, cmds))
    if verbose_ptxas:
        sys.stderr.write("".join(logs))
    if library:
        _link(LIB, [nvcc, GENCODE, "-shared", *objs])
    if binding:
        try:
            _link(BINDING, ["g++", "-shared", bind.result(), f"-L{LIBDIR}", f"-L{os.path.join(_torch_dir(), 'lib')}", "-lckv",
                            "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"])
            with open(BINDING_OF, "w") as f:
                f.write(_torch_build())
        except (OSError, RuntimeError) as e:
            if os.path.exists(BINDING):
                os.remove(BINDING)  # another torch's, or another library's
            warnings.warn(f"the tensor binding of the serving-step calls was not built: {e}")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
