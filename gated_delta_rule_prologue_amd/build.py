"""Build libprism.so (HIP for gfx950) in-tree with hipcc.

Each source compiles to an object under ``_build/`` in parallel, then the
objects link into ``gated_delta_rule_prologue_amd/libprism.so``.  The library
exports only the C ABI of ``include/prism.h`` and needs hipcc alone.  The Python calls
of the layer operators (``csrc/torch_calls.cpp``) build into ``_calls.so`` beside it, a
CPython module linked to it and to torch, where torch can be imported.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

try:
    from . import check_isa
except ImportError:                      # run as a script
    import check_isa

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libprism.so")
CALLS = os.path.join(PKG, "_calls.so")
SOURCES = ["prism_api.hip", "prologue.hip", "prologue_bf16.hip", "prologue_f32.hip",
           "prologue_bf16_ext.hip", "prologue_f32_ext.hip", "chunk_scan.hip",
           "chunk_scan_bf16.hip", "decode.hip", "long_seq.hip", "backward.hip",
           "scan_f32_recurrent.hip", "chunk_gram.hip", "chunk_scan_state.hip",
           "backward_chunk.hip", "layer_api.hip", "norm_residual.hip", "norm_gate.hip",
           "draft.hip", "verify.hip", "stack_api.hip", "short_conv.hip", "qk_norm.hip", "sample.hip"]
CHECKED = ["chunk_scan_bf16.hip", "chunk_scan.hip", "backward.hip", "chunk_gram.hip",
           "chunk_scan_state.hip", "backward_chunk.hip", "draft.hip"]   # MFMA chains, DPP
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # packed fp32 VALU ops are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA accumulators in ordinary VGPRs: the scan kernels post-process every
    # accumulator tile with VALU code, which would otherwise copy through AGPRs
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-Wall", "-Wno-unused-function",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "hipcc"


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in r.stdout.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{out}")
    if verbose and out.strip():
        print(out, flush=True)


def _torch():
    """The torch module, or None where there is none."""
    try:
        import torch
    except (ImportError, OSError):                 # OSError: a library that torch loads is missing
        return None
    return torch


def _calls_cmd(torch, out: str, link: bool):
    """Compile (or link) torch_calls.cpp: host code only."""
    torch_dir = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "torch_calls.o")
    if not link:
        inc = [INCLUDE, os.path.join(torch_dir, "include"), sysconfig.get_paths()["include"],
               os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")]
        abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
        return ["g++", "-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
                f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *("-isystem" + d for d in inc), "-Wall", "-c",
                os.path.join(CSRC, "torch_calls.cpp"), "-o", obj]
    return ["g++", "-shared", obj, "-o", out, LIB, "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN"]


def build(verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hipcc = _hipcc()
    objs = []
    cmds = []
    for src in SOURCES:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        cmds.append([hipcc, *HIPCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj])
    # device assembly of the MFMA kernels, for the machine-code check below
    asm = {src: os.path.join(BUILD, os.path.splitext(src)[0] + ".s") for src in CHECKED}
    for src, out in asm.items():
        cmds.append([hipcc, *HIPCC_FLAGS, *extra_flags, "-S", "--cuda-device-only",
                     os.path.join(CSRC, src), "-o", out])
    torch = _torch()
    with ThreadPoolExecutor(max_workers=len(cmds) + 1) as ex:
        calls = ex.submit(lambda: _run(_calls_cmd(torch, CALLS, link=False), verbose)) if torch else None
        list(ex.map(lambda c: _run(c, verbose), cmds))
    for src, out in asm.items():
        text = open(out).read()
        bad = check_isa.scan(text)
        if bad:
            lines = "\n".join(f"  {f[:70]}: {i}" for f, i in bad[:10])
            raise RuntimeError(f"{src}: a 16x16x16 MFMA overlaps the result of an in-flight "
                               f"16x16x32 MFMA (see check_isa.py):\n{lines}")
        bad = check_isa.scan_dpp(text)
        if bad:
            lines = "\n".join(f"  {f[:70]}: {i}" for f, i in bad[:10])
            raise RuntimeError(f"{src}: a DPP source is read fewer than two wait states after "
                               f"its VALU write (see check_isa.py):\n{lines}")
    tmp = LIB + ".tmp%d" % os.getpid()
    _run([hipcc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,-soname,libprism.so", *objs,
          "-o", tmp], verbose)
    os.replace(tmp, LIB)
    if os.path.exists(CALLS):                      # an earlier one may not fit the new library
        os.remove(CALLS)
    if calls is None:
        print("torch cannot be imported: _calls.so (the Python calls of the layer operators) is not built",
              flush=True)
        return LIB
    calls.result()
    tmp = CALLS + ".tmp%d" % os.getpid()
    _run(_calls_cmd(torch, tmp, link=True), verbose)
    os.replace(tmp, CALLS)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
