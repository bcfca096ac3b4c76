"""Build libsherry.so (gfx950) in-tree with hipcc, and with g++ the Python
module that marshals the feed-forward operators' tensors.

    python -m bit_weight_amd.build

Every HIP source under csrc/ is compiled for gfx950 only (one object each,
in parallel) and linked into bit_weight_amd/libsherry.so.  Packed-FP32
instruction selection is switched off for device code (-packed-fp32-ops);
hipcc's host pass warns that it does not know that feature, which is
harmless.  MFMA accumulators are kept in arch VGPRs (-amdgpu-mfma-vgpr-form).
"""

from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsherry.so")
SOURCES = ["sherry_abi.hip", "pack.hip", "lut_gemv.hip", "mfma_gemm.hip", "mfma_gemv.hip", "input_grad.hip", "norm.hip", "probe.hip",
           "head_norm.hip", "kv_cache.hip", "cache_attention.hip", "cache_attention_tiles.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]
# MFMA accumulators in arch VGPRs: the matrix ops then accumulate in place
# instead of shuffling accumulation registers every k-step
VGPR_FORM = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
# Kernel arguments preloaded into SGPRs at dispatch instead of read from the
# kernel-argument segment by the first instructions: the product kernels'
# eight leading ones (packed, x, xf, M, N, K and two plan integers, 11
# SGPRs), the quantizer's four (x, q, s_x, K)
PRELOAD = {"mfma_gemv.hip": ["-mllvm", "-amdgpu-kernarg-preload-count=8"],
           "lut_gemv.hip": ["-mllvm", "-amdgpu-kernarg-preload-count=8"],
           "mfma_gemm.hip": ["-mllvm", "-amdgpu-kernarg-preload-count=8"],
           "pack.hip": ["-mllvm", "-amdgpu-kernarg-preload-count=4"]}


# The Python module (host code only): torch's headers and libraries, and the
# library's functions by address
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_binding.so")


def binding_command(out: str) -> list[str]:
    import torch

    root = os.path.dirname(torch.__file__)
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"), sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f"-I{d}" for d in include], BINDING_SOURCE, "-o", out, f"-L{os.path.join(root, 'lib')}",
            "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python"]


def _filter(text: str) -> str:
    return "\n".join(l for l in text.splitlines() if "packed-fp32-ops" not in l)


def build(verbose: bool = False) -> str:
    """Compile every source into libsherry.so and _binding.so (always recompiles)."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory(prefix="sherry_build_") as obj_dir:
        procs = []
        for src in SOURCES:
            obj = os.path.join(obj_dir, src.replace(".hip", ".o"))
            cmd = [HIPCC, *FLAGS, *VGPR_FORM, *PRELOAD.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                     stderr=subprocess.STDOUT, text=True)))
        cmd = binding_command(BINDING + ".tmp")
        if verbose:
            print(" ".join(cmd), flush=True)
        binding = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        objs = []
        for src, obj, proc in procs:
            out = _filter(proc.communicate()[0])
            if proc.returncode != 0:
                raise RuntimeError(f"hipcc failed on {src} ({proc.returncode}):\n{out}")
            if verbose and out.strip():
                print(out, flush=True)
            objs.append(obj)
        cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed ({res.returncode}):\n{_filter(res.stdout + res.stderr)}")
        out = binding.communicate()[0]
        if binding.returncode != 0:
            raise RuntimeError(f"g++ failed on binding.cpp ({binding.returncode}):\n{out}")
    os.replace(tmp, LIB)
    os.replace(BINDING + ".tmp", BINDING)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
