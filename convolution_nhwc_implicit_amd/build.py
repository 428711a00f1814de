"""Build the HIP library (libconv2d_nhwc.so) for gfx950 and the sequence
operators' binding to torch tensors (_sequence.so), in-tree.

    python -m convolution_nhwc_implicit_amd.build

Every source under csrc/ is compiled by hipcc for --offload-arch=gfx950 and
linked into one shared library next to this file.  Packed fp32 instructions
are disabled for all device code.  The binding is host code against torch's
headers, compiled by g++ and linked to that library beside it.
"""
import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libconv2d_nhwc.so")
BINDING = os.path.join(PKG, "_sequence.so")
ARCH = "gfx950"

SOURCES = ["api.cpp", "igemm.hip", "band.hip", "wino.hip", "wgrad.hip", "wgrad_band.hip", "direct.hip", "repack.hip", "fewchan.hip", "fewchan_wgrad.hip", "fewchan_dgrad.hip", "pointwise.hip", "pointwise_wgrad.hip", "patch.hip",
           "seq_api.cpp", "causal_conv.hip", "selective_scan.hip", "selective_scan_grad.hip",
           "fp8_quantize.hip", "fp8_matmul.hip"]

COMMON_FLAGS = [
    "-x", "hip", f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Wall", "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def hipcc():
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found: the HIP toolchain is required to build the library")
    return path


def rocm_path():
    return os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))


def _compile(src, extra):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc()] + COMMON_FLAGS + list(extra) + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{msg}")
    return obj, msg


def _compile_binding():
    import torch

    top = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "seq_binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
           "-isystem", os.path.join(top, "include"),
           "-isystem", os.path.join(top, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(rocm_path(), "include"),
           "-c", os.path.join(CSRC, "seq_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for seq_binding.cpp:\n" + r.stdout + r.stderr)
    return obj, r.stderr, os.path.join(top, "lib")


def _link(cmd, out):
    tmp = out + ".tmp%d" % os.getpid()
    r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, out)


def build(verbose=False, extra_flags=()):
    """Compile all sources and link libconv2d_nhwc.so and _sequence.so.  Always rebuilds."""
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(lambda s: _compile(s, extra_flags), SOURCES))
        bind_obj, bind_msg, torch_lib = binding.result()
    for obj, msg in results:
        if verbose and msg.strip():
            print(msg, file=sys.stderr)
    _link([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC"] + [o for o, _ in results], LIB)
    if verbose and bind_msg.strip():
        print(bind_msg, file=sys.stderr)
    _link(["g++", "-shared", "-fPIC", bind_obj, f"-L{PKG}", "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
           f"-L{torch_lib}", "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python"], BINDING)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
