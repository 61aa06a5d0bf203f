"""Build libgemm_f32.so, and the Python module _expert_binding in front of its
expert-layer entry points, in-tree with hipcc for gfx950.

Usage: ``python -m dense_gemm_optimisation_fp32_amd.build`` (or call
``build()``).  Always recompiles.

The kernels are compiled in several translation units in parallel
(``csrc/k_*.hip``, explicit instantiations of the lists in
``csrc/kernel_list.hpp``, and the expert-layer kernels with their launches);
the host units ``csrc/gemm_f32.hip`` and ``csrc/expert_ops.hip`` hold the C ABI
and only take the kernels' handles.  The compiler's per-kernel resource
report (VGPRs, AGPRs, SGPRs, LDS, scratch, occupancy) is kept in
``_build/kernel_resources.txt`` for the tile/occupancy sweep and compiled into
the library as a table (``_build/kernel_resources.cpp``), which
``gemm_f32_describe`` and ``gemm_f32_variant_info`` report from.
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
LIB_PATH = os.path.join(PKG_DIR, "libgemm_f32.so")
BINDING_SOURCE = os.path.join(CSRC, "expert_binding.cpp")
BINDING_PATH = os.path.join(PKG_DIR, "_expert_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILD_DIR = os.path.join(PKG_DIR, "_build")
HOST_SOURCES = [os.path.join(CSRC, "gemm_f32.hip"), os.path.join(CSRC, "expert_ops.hip")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-mcode-object-version=5",
    # Packed FP32 instructions stay off in every kernel.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]
REMARKS = "-Rpass-analysis=kernel-resource-usage"


def kernel_sources():
    return sorted(glob.glob(os.path.join(CSRC, "k_*.hip")))


def parse_resources(text: str):
    """The compiler's resource remarks: [(mangled name, {field: value})]."""
    out = []
    cur = None
    for line in text.splitlines():
        m = re.search(r"remark:\s+([A-Za-z /\[\]]+?):\s+(\S+)", line)
        if not m:
            continue
        key, val = m.group(1).strip(), m.group(2)
        if key == "Function Name":
            cur = {}
            out.append((val, cur))
        elif cur is not None:
            cur[key] = val
    return out


def resource_table_source(entries) -> str:
    rows = []
    for name, r in sorted(entries):
        vals = [int(r.get(f, 0)) for f in ("VGPRs", "AGPRs", "TotalSGPRs", "ScratchSize [bytes/lane]",
                                            "LDS Size [bytes/block]", "Occupancy [waves/SIMD]")]
        rows.append('    {"%s", %s},' % (name, ", ".join(str(v) for v in vals)))
    return ("// Generated by build.py from the compiler's resource report; not edited by hand.\n"
            '#include "kernel_resources.hpp"\n\nnamespace gemmf32 {\n\n'
            "const KernelResources kKernelResources[] = {\n" + "\n".join(rows) + "\n};\n"
            f"const int kKernelResourcesCount = {len(rows)};\n\n}}  // namespace gemmf32\n")


def _compile_all(jobs, verbose):
    """Run (cmd, log) jobs in parallel; return {log: (returncode, stderr)}."""
    procs = []
    for cmd, log in jobs:
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True), log))
    out = {}
    for p, log in procs:
        _, err = p.communicate()
        out[log] = (p.returncode, err)
    return out


def _fail(what, err):
    errors = [ln for ln in err.splitlines() if "error" in ln or "Error" in ln]
    raise RuntimeError(f"{what} failed:\n" + "\n".join(errors[:40] or err.splitlines()[-40:]))


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    inc = ["-I", INCLUDE, "-I", CSRC]
    jobs = []
    objs = []
    for src in kernel_sources() + HOST_SOURCES:
        obj = os.path.join(BUILD_DIR, os.path.basename(src).replace(".hip", ".o"))
        objs.append(obj)
        jobs.append(([HIPCC, *HIPCC_FLAGS, *inc, REMARKS, "-c", "-o", obj, src], src))
    results = _compile_all(jobs, verbose)

    report = []
    entries = []
    for src in kernel_sources() + HOST_SOURCES:
        rc, err = results[src]
        report.append(err)
        if rc != 0:
            _fail(f"hipcc {os.path.basename(src)}", err)
        found = parse_resources(err)
        if src in HOST_SOURCES and found:
            raise RuntimeError("kernels instantiated in a host unit (instantiate them in a kernel unit): "
                               + ", ".join(n for n, _ in found[:5]))
        entries.extend(found)
    with open(os.path.join(BUILD_DIR, "kernel_resources.txt"), "w") as f:
        f.write("".join(report))

    table_src = os.path.join(BUILD_DIR, "kernel_resources.cpp")
    with open(table_src, "w") as f:
        f.write(resource_table_source(entries))
    table_obj = os.path.join(BUILD_DIR, "kernel_resources.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", CSRC, "-c", "-o", table_obj, table_src]
    if verbose:
        print(" ".join(cmd), flush=True)
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        _fail("resource table", p.stderr)

    tmp = LIB_PATH + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs, table_obj, "-ldl"]
    if verbose:
        print(" ".join(cmd), flush=True)
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        _fail("link", p.stderr)
    os.replace(tmp, LIB_PATH)

    build_binding(verbose)
    return LIB_PATH


def build_binding(verbose: bool = False) -> None:
    """The Python module in front of the expert-layer entry points.  The library
    itself needs neither Python's nor torch's C++ headers: where they are not
    installed it stays without the module, which the operators then name as
    missing when they are called."""
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    include = os.path.join(os.path.dirname(torch.__file__), "include")
    python_include = sysconfig.get_paths()["include"]
    missing = [h for h in (os.path.join(python_include, "Python.h"), os.path.join(include, "torch", "csrc", "Exceptions.h"))
               if not os.path.exists(h)]
    if missing:
        if os.path.exists(BINDING_PATH):
            os.remove(BINDING_PATH)
        print(f"{os.path.basename(BINDING_PATH)} is not built: no {', '.join(missing)}", file=sys.stderr)
        return
    tmp = BINDING_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-isystem", python_include, "-o", tmp, BINDING_SOURCE,
           "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        _fail("expert_binding.cpp", p.stderr)
    os.replace(tmp, BINDING_PATH)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
