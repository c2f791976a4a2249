"""Compile the HIP library ``libconv_bn_silu.so`` for gfx950 and the Python
module ``_block8.so`` that calls it (both in-tree).

Every ``csrc/*.hip`` and ``csrc/*.cpp`` but ``py_*.cpp`` is compiled by hipcc to its own object
(in parallel) and linked into one shared library next to this file.  All HIP
code is compiled without packed-fp32 instructions.

The compiler's per-kernel resource report (registers, LDS, scratch) is written
to ``libconv_bn_silu.resources.txt`` beside the library, and the build fails if
a kernel needs scratch memory: register spills or an array the compiler could
not keep in registers turn the kernel's hot loop into memory traffic (one such
kernel ran six times slower than without), so they are treated as errors.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libconv_bn_silu.so")
RESOURCES = os.path.join(HERE, "libconv_bn_silu.resources.txt")
MODULE = os.path.join(HERE, "_block8.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

COMMON = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I" + os.path.join(HERE, "..", "include")]


def sources():
    cpp = [s for s in glob.glob(os.path.join(CSRC, "*.cpp")) if not os.path.basename(s).startswith("py_")]
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")) + cpp)


_REMARK = re.compile(r"remark:\s+(Function Name|VGPRs|AGPRs|ScratchSize \[bytes/lane\]|Occupancy \[waves/SIMD\]|"
                     r"LDS Size \[bytes/block\]|VGPRs Spill|SGPRs Spill):\s*(\S+)")


def parse_resources(text: str) -> list[dict]:
    """Per-kernel records from hipcc's kernel-resource-usage remarks."""
    out: list[dict] = []
    for line in text.splitlines():
        m = _REMARK.search(line)
        if not m:
            continue
        key, val = m.group(1), m.group(2)
        if key == "Function Name":
            out.append({"kernel": val})
        elif out:
            out[-1][key.split(" [")[0]] = int(val)
    return out


def _compile(src: str, extra: list[str]) -> tuple[str, list[dict]]:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC] + COMMON + extra + ["-Rpass-analysis=kernel-resource-usage", "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed on {os.path.basename(src)}")
    # hipcc's host pass does not know the packed-fp32 feature and says so;
    # print only other diagnostics (not the resource remarks either).
    other = [l for l in res.stderr.splitlines()
             if "packed-fp32-ops" not in l and "-Rpass-analysis=kernel-resource-usage" not in l]
    if other:
        sys.stderr.write("\n".join(other) + "\n")
    return obj, parse_resources(res.stderr)


def _module_needs() -> tuple[str, list[str]]:
    """PyTorch's folder, and what of the module's needs is not there."""
    spec = importlib.util.find_spec("torch")
    root = os.path.dirname(spec.origin) if spec and spec.origin else ""
    needs = {"PyTorch with its headers": os.path.join(root, "include", "ATen", "core", "Tensor.h"),
             "Python's headers": os.path.join(sysconfig.get_paths()["include"], "Python.h")}
    missing = [what for what, path in needs.items() if not os.path.exists(path)]
    return root, missing + ([] if shutil.which("g++") else ["g++"])


def build_module() -> str | None:
    """The Python module: host code only, against PyTorch's headers and the library.  Where those or
    g++ are absent there is none (and the library, which needs neither, is whole without it): then
    the 8-bit block operators are reached through the C ABI only, and importing ``block8`` fails."""
    root, missing = _module_needs()
    if missing:
        if os.path.exists(MODULE):
            os.remove(MODULE)  # of another build of the library
        sys.stderr.write(f"{os.path.basename(MODULE)} is not built: {', '.join(missing)} not found\n")
        return None
    import torch
    tmp = MODULE + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(root, "include"), "-isystem", os.path.join(root, "include/torch/csrc/api/include"),
           "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"],
           *sorted(glob.glob(os.path.join(CSRC, "py_*.cpp"))), "-o", tmp, "-L" + HERE, "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(root, "lib"),
           "-l:libconv_bn_silu.so", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, MODULE)
    return MODULE


def build(extra: list[str] | None = None, jobs: int = 8) -> str:
    """Compile and link; returns the path of the shared library."""
    os.makedirs(BUILD, exist_ok=True)
    extra = list(extra or [])
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        done = list(ex.map(lambda s: _compile(s, extra), sources()))
    objs = [o for o, _ in done]
    kernels = [k for _, ks in done for k in ks]
    with open(RESOURCES, "w") as f:
        f.write("# kernel  VGPRs  AGPRs  scratch_bytes_per_lane  LDS_bytes  waves_per_SIMD\n")
        for k in kernels:
            f.write(f"{k['kernel']}  {k.get('VGPRs')}  {k.get('AGPRs')}  {k.get('ScratchSize')}  "
                    f"{k.get('LDS Size')}  {k.get('Occupancy')}\n")
    spilling = [k["kernel"] for k in kernels if k.get("ScratchSize", 0) or k.get("VGPRs Spill", 0)]
    if spilling:
        raise RuntimeError("kernels using scratch memory: " + ", ".join(spilling))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_module()
    return LIB


if __name__ == "__main__":
    print(build())
