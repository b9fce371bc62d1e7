"""Builds the library ``_build/libawq_gb300.so`` in-tree with nvcc for sm_103a.

Every ``csrc/*.cu`` translation unit is compiled in parallel, then linked
into one shared library with the CUDA runtime linked statically. Rebuilds
only what is older than its sources (any header change rebuilds all units).

It also builds ``_build/libawq_gb300_fault_test.so``, the fault-test build
used only by the tests: the units with bounded device waits (the C ABI, the
decode, prefill and attention kernels) compiled again with ``-DAWQ_FAULT_TEST`` (a wait
limit of about 2 ms and the switch declared in
``include/awq_gb300_fault_test.h``), linked with the other units' objects.

And ``_build/awq_step-<torch version>-<interpreter>.so``, the Python module behind ``step.py``
(``csrc/awq_step_module.cpp``, compiled with the host compiler against the
installed torch).

    python -m bit_weight_quantized_awq_gb300.build [--force] [--ptxas-verbose]
"""
from __future__ import annotations

import argparse
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

from ._binding import STEP_PATH as STEP_MODULE

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libawq_gb300.so")
FAULT_LIB = os.path.join(BUILD, "libawq_gb300_fault_test.so")
FAULT_BUILD = os.path.join(BUILD, "fault_test")
# units whose kernels wait on barriers or flags (and the ABI that sets the switch)
FAULT_UNITS = ("awq_api.cu", "awq_decode.cu", "awq_prefill.cu", "awq_attention.cu", "awq_attention_tc.cu")
INCLUDE = os.path.join(ROOT, "include")
STEP_SOURCE = os.path.join(CSRC, "awq_step_module.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the AWQ library needs the CUDA toolkit to build")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _fault_obj(src: str) -> str:
    return os.path.join(FAULT_BUILD, os.path.basename(src)[:-3] + ".o")


def _step_command(out: str) -> list[str]:
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        raise RuntimeError("g++ not found: the AWQ step module needs a host compiler to build")
    include = [sysconfig.get_paths()["include"], INCLUDE, os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")]
    # torch has loaded its libraries by the time that the module is
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", *(f"-I{d}" for d in include), STEP_SOURCE, "-o", out,
            "-L" + os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(FAULT_BUILD, exist_ok=True)
    cc = nvcc()
    headers = _headers()
    jobs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if force or _stale(obj, [src] + headers + [os.path.abspath(__file__)]):
            cmd = [cc] + ARCH + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + \
                  ["-c", src, "-o", obj]
            jobs.append((src, cmd))
        if os.path.basename(src) in FAULT_UNITS:
            fobj = _fault_obj(src)
            if force or _stale(fobj, [src] + headers + [os.path.abspath(__file__)]):
                jobs.append((src + " (fault test)", [cc] + ARCH + NVCC_FLAGS + ["-DAWQ_FAULT_TEST", "-c", src,
                                                                               "-o", fobj]))
    library_jobs = bool(jobs)
    step_tmp = STEP_MODULE + f".tmp{os.getpid()}"
    if force or _stale(STEP_MODULE, [STEP_SOURCE, os.path.join(INCLUDE, "awq_gb300.h"), os.path.abspath(__file__)]):
        jobs.append((STEP_SOURCE, _step_command(step_tmp)))
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in _sources()]
    fault_objs = [_fault_obj(s) if os.path.basename(s) in FAULT_UNITS else
                  os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in _sources()]

    def run(job):
        src, cmd = job
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, r

    failed = []
    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for src, r in ex.map(run, jobs):
                if r.returncode != 0:
                    failed.append((src, r.stderr))
                elif (ptxas_verbose or r.stderr.strip()) and not quiet:
                    sys.stderr.write(r.stderr)
    if failed:
        msg = "\n".join(f"--- {s}\n{e}" for s, e in failed)
        raise RuntimeError(f"compilation failed:\n{msg}")
    if os.path.exists(step_tmp):
        os.replace(step_tmp, STEP_MODULE)
    for lib, lib_objs in ((LIB, objs), (FAULT_LIB, fault_objs)):
        if force or library_jobs or _stale(lib, lib_objs):
            tmp = lib + f".tmp{os.getpid()}"
            cmd = [cc] + ARCH + ["-shared", "-o", tmp] + lib_objs
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stderr}")
            os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.ptxas_verbose))
