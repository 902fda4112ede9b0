"""Build libmla_decode.so in-tree with nvcc for sm_103a (no cmake, no torch). Where
PyTorch is there, also the compiled Python binding of the prefill step's calls (the
host compiler, PyTorch's headers), in a file named after the versions that it is for.

Each .cu file compiles to an object in parallel; the objects link into one
shared library with the CUDA runtime linked statically, so the library loads
on a machine without a GPU driver (the exported symbols can be inspected
there; calling them needs a GPU).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmla_decode.so")
SOURCES = ["mla_api.cu", "kv_write.cu", "plan_merge.cu", "decode_sm103.cu", "uv_project.cu", "selftest.cu",
           "step_api.cu", "step_tables.cu", "rope_write.cu", "prefill_gather.cu", "prefill_expand.cu", "prefill_attn.cu",
           "prefill_absorb.cu", "shared_api.cu", "shared_plan.cu", "shared_decode.cu", "quant_store.cu"]
HEADERS = ["ptx.cuh", "mla_internal.h", "trace.cuh", "host_util.h", "step_internal.h", "ptx_prefill.cuh", "scan.cuh",
           "shared_internal.h", "ptx_shared.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _deps():
    inc = os.path.join(os.path.dirname(HERE), "include", "mla_decode.h")
    return [os.path.join(CSRC, h) for h in HEADERS] + [inc, os.path.abspath(__file__)]


def _stale(target, inputs):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(i) > t for i in inputs)


def _run(cmd) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compiler failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    return r.stderr


def binding_path() -> str:
    """The binding for this Python and this PyTorch (their ABIs change between versions)."""
    import torch
    return os.path.join(HERE, "_step_binding.%s-torch%s.so" % (sys.implementation.cache_tag, torch.__version__))


def _binding_command(target: str):
    import torch
    root = os.path.dirname(torch.__file__)
    dirs = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(os.path.dirname(nvcc()), "..", "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
            *[x for d in dirs for x in ("-isystem", d)], os.path.join(CSRC, "step_binding.cpp"), "-o", target,
            "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _make_binding(target: str) -> None:
    tmp = target + ".tmp.%d" % os.getpid()
    _run(_binding_command(tmp))
    os.replace(tmp, target)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False, defines=(),
          lib_path: str = LIB, build_dir: str = BUILD) -> str:
    """Compile every kernel file, link libmla_decode.so and build the binding (only what is stale).
    `defines` (e.g. ["-DMLA_TRACE"] for the event-traced build) go with
    their own lib_path and build_dir. The library does not wait for the binding: it is there
    even where the binding could not be made (an error) or PyTorch is missing (none)."""
    os.makedirs(build_dir, exist_ok=True)
    deps = _deps()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
                    "--expt-relaxed-constexpr", *defines]
    if ptxas_info:
        flags += ["-Xptxas", "-v"]
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(build_dir, src.replace(".cu", ".o"))
        objs.append(o)
        if force or ptxas_info or _stale(o, [s] + deps):
            jobs.append([nvcc(), *flags, "-c", s, "-o", o])

    binding = None
    if lib_path == LIB:
        try:
            binding = binding_path()
        except ImportError:
            pass
    if binding and not force and not _stale(binding, [os.path.join(CSRC, "step_binding.cpp")] + deps[-2:]):
        binding = None

    with cf.ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
        made = ex.submit(_make_binding, binding) if binding else None
        for log in ex.map(_run, jobs):
            if verbose and log:
                print(log)
        if force or jobs or _stale(lib_path, objs):
            tmp = lib_path + ".tmp.%d" % os.getpid()
            _run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"])
            os.replace(tmp, lib_path)
        if made:
            try:
                made.result()
            except (RuntimeError, OSError) as e:
                raise RuntimeError("%s is built, its Python binding is not: %s" % (os.path.basename(lib_path), e)) from e
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
