"""Builds ``librgdr.so`` (the gfx950 HIP library behind ``include/rgdr.h``) and ``_la_binding.so``
(a CPython module, host code only, linked against torch) in-tree.

    python -m gated_delta_rule_rgdr_amd.build [--verbose]

Every source is compiled for gfx950 only. Packed fp32 instructions are switched off for
device code (``-target-feature -packed-fp32-ops``); the host pass prints a harmless
warning that it does not know that feature.
"""
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "librgdr.so")
BINDING = os.path.join(PKG, "_la_binding.so")

SOURCES = ["rgdr_decode.hip", "rgdr_prefill.hip", "la_gate.hip", "la_decode.hip",
           "la_prefill.hip", "la_state.hip", "la_norm_gate.hip", "la_conv.hip", "la_rope.hip",
           "ssm_decode.hip", "ssm_prefill.hip", "rgdr_host.cpp"]
ARCH = "gfx950"
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def compile_cmd(src, obj, extra=()):
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    return (["hipcc", f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall"]
            + DEVICE_FLAGS + ["-I", INCLUDE, "-I", CSRC] + lang + list(extra)
            + ["-c", src, "-o", obj])


def binding_cmds(obj):
    """Compile and link commands of the CPython module."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    include = [sysconfig.get_paths()["include"], *cpp_extension.include_paths(),
               os.path.join(rocm, "include"), INCLUDE]
    compile_ = (["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
                 f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
                + [x for d in include for x in ("-isystem", d)]
                + ["-c", os.path.join(CSRC, "la_binding.cpp"), "-o", obj])
    link = ["g++", "-shared", "-fPIC", obj, "-L", PKG, "-l:librgdr.so", "-L", lib, "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}", "-o", BINDING + ".tmp"]
    return compile_, link


def _finish(procs, verbose):
    """The sources whose compilation failed."""
    failed = []
    for s, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        # the host pass's note about the device-only feature is expected noise
        lines = [ln for ln in text.splitlines() if "packed-fp32-ops" not in ln]
        if lines and (verbose or p.returncode):
            print("\n".join(lines), file=sys.stderr)
        if p.returncode:
            failed.append(s)
    if failed:
        raise RuntimeError(f"the compiler failed for {failed}")


def build(verbose: bool = False, extra=()) -> str:
    """Both libraries. ``librgdr.so`` needs neither Python's nor torch's headers and is in place when
    an error of the other one is raised."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = []
    objs = []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(BUILD_DIR, os.path.splitext(s)[0] + ".o")
        cmd = compile_cmd(src, obj, extra)
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((s, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    _finish(procs, verbose)
    tmp = LIB + ".tmp"
    link = ["hipcc", f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    if verbose:
        print(" ".join(link), flush=True)
    subprocess.run(link, check=True)
    os.replace(tmp, LIB)
    build_binding(verbose)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """The CPython module, against a built ``librgdr.so``."""
    obj = os.path.join(BUILD_DIR, "la_binding.o")
    compile_, link = binding_cmds(obj)
    if verbose:
        print(" ".join(compile_), flush=True)
    _finish([("la_binding.cpp", subprocess.Popen(compile_, stdout=subprocess.PIPE,
                                                 stderr=subprocess.STDOUT))], verbose)
    if verbose:
        print(" ".join(link), flush=True)
    subprocess.run(link, check=True)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))
