"""Build libskinny.so in-tree with hipcc for gfx950, and _binding.so, the Python
extension that checks torch tensors for some of its calls, against the torch in use.
Where torch cannot be imported the library alone is built.

    python -m fp8_quantized_skinny_amd.build

Every HIP source is compiled with packed-fp32 instructions disabled
(-Xclang -target-feature -Xclang -packed-fp32-ops): the kernels get no
v_pk_*_f32 from the compiler.

The build also reads the compiler's per-kernel resource report and fails if a
kernel spills registers to scratch memory beyond KNOWN_SPILLS: a spill turns
the kernels' exact per-chunk load waits into full waits, so it is a
performance regression even when results stay right.
"""

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libskinny.so")
BINDING = os.path.join(PKG, "_binding.so")
SOURCES = ["host.cpp", "nvfp4_gemm.hip", "fp8_gemm.hip", "reduce.hip", "probe.hip", "noalloc.hip",
           "kv4_host.cpp", "kv4_cache.hip", "kv4_attention.hip", "kv4_chunk.hip", "rope.hip", "logprobs.hip"]
ARCH = "gfx950"

# Kernels known to spill, with their scratch bytes per lane: the streaming
# lm_head instance for three K spans (K <= 3072), which no decode shape here
# uses.
KNOWN_SPILLS = {"_ZN6skinny12_GLOBAL__N_112nvfp4_streamILi3ELi1EEEvNS0_9Nvfp4ArgsE": 24}


def hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def build(verbose=False):
    """Build libskinny.so and, if torch can be imported, _binding.so; returns the library path."""
    build_library(verbose)
    try:
        import torch  # noqa: F401
    except ImportError:  # host-only use (packing, quantizing): nothing calls the binding
        return LIB
    build_binding(verbose)
    return LIB


def build_library(verbose=False):
    """Compile every source and link libskinny.so; returns the library path."""
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    common = ["-O3", "-std=c++17", "-fPIC", "-pthread", "-Wall", "-I", INCLUDE, "-I", CSRC]
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src + ".o")
        cmd = [hipcc(), *common, "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".hip"):
            cmd[1:1] = ["-x", "hip", f"--offload-arch={ARCH}",
                        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                        "-Rpass-analysis=kernel-resource-usage"]
        out = _run(cmd, verbose)
        if src.endswith(".hip"):
            check_spills(scratch_per_kernel(out), src)
        objs.append(obj)
    tmp = LIB + ".tmp"
    _run([hipcc(), "-shared", "-fPIC", "-pthread", f"--offload-arch={ARCH}", *objs, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


def build_binding(verbose=False):
    """Compile csrc/binding.cpp against torch's headers; it finds libskinny.so beside itself."""
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    include = [INCLUDE, os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               os.path.join(rocm, "include"), sysconfig.get_paths()["include"]]
    tmp = BINDING + ".tmp"
    _run([hipcc(), "-no-hip-rt", "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
          "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", f'-DSKINNY_TORCH_VERSION="{torch.__version__}"',
          *[f"-I{i}" if i == INCLUDE else f"-isystem{i}" for i in include], os.path.join(CSRC, "binding.cpp"), "-o", tmp,
          "-L" + PKG, "-l:libskinny.so", "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(home, "lib"),
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"], verbose)
    os.replace(tmp, BINDING)
    return BINDING


def scratch_per_kernel(report):
    """{kernel symbol: scratch bytes per lane} from the compiler's
    kernel-resource-usage remarks."""
    import re
    sizes, name = {}, None
    for line in report.splitlines():
        m = re.search(r"remark: Function Name: (\S+)", line)
        if m:
            name = m.group(1)
            continue
        m = re.search(r"remark:\s+ScratchSize \[bytes/lane\]: (\d+)", line)
        if m and name:
            sizes[name] = int(m.group(1))
    return sizes


def check_spills(sizes, src):
    bad = {k: v for k, v in sizes.items() if v > KNOWN_SPILLS.get(k, 0)}
    if bad:
        raise RuntimeError(f"build failed: {src}: kernels spill to scratch (bytes per lane): {bad}")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in r.stdout.splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"build failed: {' '.join(cmd)}\n{out}")
    if verbose and out.strip():
        print("\n".join(l for l in out.splitlines() if "kernel-resource-usage" not in l))
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
