"""Build the PN CUDA library in-tree: ``bit_weight_only_pn_gb300/libpn_gb300.so``.

Each translation unit in ``csrc/`` is compiled for sm_103a in parallel, then
linked into one shared library with the CUDA runtime linked statically, so the
library loads without any other CUDA shared object.  The Python entry of the
serving-step calls (``_step.so``, plain C++ against PyTorch's headers) is built
beside it.  Objects go to ``bit_weight_only_pn_gb300/_build/``.  Rebuilds only
what is out of date.
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
LIBRARY = os.path.join(HERE, "libpn_gb300.so")
BINDING = os.path.join(HERE, "_step.so")
SOURCES = ["pn_attn.cu", "pn_attn_tc.cu", "pn_capi.cu", "pn_codec.cu", "pn_gemv_ffma.cu", "pn_gemv_simt.cu", "pn_gemv_stream.cu", "pn_gemv_tc.cu",
           "pn_gptq.cu", "pn_kv.cu", "pn_noalloc.cu", "pn_prefill.cu", "pn_probe.cu", "pn_rotate.cu", "pn_verify.cu"]
HEADERS = ["pn_attn.cuh", "pn_device.cuh", "pn_internal.h", "pn_kv.cuh", "pn_tcgen05.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, extra=()) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    deps = [os.path.join(CSRC, src)] + [os.path.join(CSRC, h) for h in HEADERS] + \
        [os.path.join(ROOT, "include", "pn.h")]
    if _newer(obj, deps):
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    return obj


def _run(cmd, what: str) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")


def _torch():
    """PyTorch's include folders, library folder, version and C++ ABI flag."""
    import torch
    root = os.path.dirname(torch.__file__)
    include = os.path.join(root, "include")
    return ([include, os.path.join(include, "torch", "csrc", "api", "include")], os.path.join(root, "lib"),
            torch.__version__, int(torch._C._GLIBCXX_USE_CXX11_ABI))


def _binding_key() -> str:
    """What the Python entry is built against: PyTorch, its C++ ABI, the Python and machine."""
    _, _, version, abi = _torch()
    return f"{version}-cxx11abi{abi}-{sysconfig.get_config_var('SOABI')}"


def _compile_binding() -> str:
    src = os.path.join(CSRC, "pn_step_binding.cpp")
    include, _, _, abi = _torch()
    # one object per PyTorch and Python: their headers are part of it
    obj = os.path.join(BUILD, f"pn_step_binding-{_binding_key()}.o")
    if _newer(obj, [src, os.path.join(ROOT, "include", "pn.h")]):
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
        _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
              *(f"-I{d}" for d in [*include, cuda, sysconfig.get_paths()["include"]]), "-c", src, "-o", obj],
             "g++ for pn_step_binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    # what the entry that lies there was built against, which its age does not tell
    record = os.path.join(BUILD, "step_binding_key.txt")
    have = None
    if os.path.exists(record):
        with open(record) as f:
            have = f.read()
    if have != _binding_key() or _newer(BINDING, [obj, LIBRARY]):
        if have is not None:
            os.remove(record)
        tmp = BINDING + ".tmp"
        _run(["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-l:" + os.path.basename(LIBRARY), f"-L{_torch()[1]}",
              "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"],
             "link of the Python entry")
        os.replace(tmp, BINDING)
        with open(record, "w") as f:
            f.write(_binding_key())


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
        binding = pool.submit(_compile_binding)
        objs = list(pool.map(_compile, SOURCES))
        binding = binding.result()
    if _newer(LIBRARY, objs):
        tmp = LIBRARY + ".tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIBRARY)
    _link_binding(binding)
    if verbose:
        print(LIBRARY)
    return LIBRARY


if __name__ == "__main__":
    build(verbose="-q" not in sys.argv)
