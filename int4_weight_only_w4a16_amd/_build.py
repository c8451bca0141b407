"""Ahead-of-time build of libw4a16.so for gfx950 with hipcc (in-tree)."""

from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libw4a16.so")
BINDING_PATH = os.path.join(PKG_DIR, "_kv4.so")

SOURCES = ("w4a16_capi.hip", "decode_gfx950.hip", "prefill_gfx950.hip", "lora_gfx950.hip",
           "probe_gfx950.hip", "kv4_capi.hip", "kv4_store_gfx950.hip", "kv4_attn_gfx950.hip",
           "kv4_prefill_gfx950.hip", "kv4_mass_gfx950.hip",
           "kv4_evict_gfx950.hip", "delta_capi.hip", "short_conv_gfx950.hip", "delta_step_gfx950.hip",
           "delta_chunk_gfx950.hip")
BINDINGS = ("kv4_binding.cpp", "delta_binding.cpp")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # no packed-fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


# Flags of single sources.
OWN_FLAGS = {
    # accumulators in ordinary registers, where other instructions take them as they are
    "delta_chunk_gfx950.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
}


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, *OWN_FLAGS.get(src, []), *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"hipcc failed on {src}")
    if extra:
        with open(os.path.join(BUILD_DIR, src + ".remarks.txt"), "w") as f:
            f.write(r.stderr)
    return obj


def _compile_binding(src: str) -> str:
    """The object of a source in BINDINGS: host code against the installed torch's headers."""
    import sysconfig

    import torch
    include = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           "-DTORCH_EXTENSION_NAME=_kv4", "-DTORCH_API_INCLUDE_EXTENSION_H",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"],
           "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"g++ failed on {src}")
    return obj


def _link_binding(objs: list[str]) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + ".tmp%d" % os.getpid()
    subprocess.run(["g++", "-shared", "-fPIC", *objs, "-o", tmp, "-L", PKG_DIR, "-l:libw4a16.so", "-L", lib, "-lc10",
                    "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN"],
                   check=True)
    os.replace(tmp, BINDING_PATH)


def build(resource_usage: bool = False) -> str:
    """Compile every HIP source for gfx950, link libw4a16.so next to this file, and build the
    operators' Python binding against it."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Rpass-analysis=kernel-resource-usage"] if resource_usage else []
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + len(BINDINGS)) as ex:
        bindings = [ex.submit(_compile_binding, s) for s in BINDINGS]
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
        bindings = [b.result() for b in bindings]
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    _link_binding(bindings)
    return LIB_PATH


if __name__ == "__main__":
    print(build(resource_usage="--resource-usage" in sys.argv))
