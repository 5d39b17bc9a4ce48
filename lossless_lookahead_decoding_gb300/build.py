"""Build liblookahead.so in-tree with nvcc for sm_103a (GB300).

Each csrc/*.cu is compiled in parallel into _build/, then linked into
lossless_lookahead_decoding_gb300/liblookahead.so against the shared CUDA
runtime.  Rebuilds only what changed (object newer than its source and every
header).  csrc/kv4_torch.cpp and kv16_torch.cpp become _kv4.so and _kv16.so,
the Python modules behind KV4Cache and KV16Cache, compiled by the host
compiler against torch's headers; without a CUDA build of torch, which the
classes need, they are left out.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "liblookahead.so")
BINDING = os.path.join(HERE, "_kv4.so")
BINDING16 = os.path.join(HERE, "_kv16.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")  # without importing it
    at = os.path.dirname(spec.origin) if spec and spec.origin else ""
    return at if os.path.exists(os.path.join(at, "include", "c10", "cuda", "CUDAStream.h")) else None


def cuda_include() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return os.path.join(home, "include")


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    hdr_t = max(os.path.getmtime(h) for h in headers)
    jobs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_t):
            jobs.append((src, obj))

    def cc(job):
        src, obj = job
        cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return r.stderr

    # the bindings' objects: as the others, with the host compiler
    torch = torch_dir()
    binding_hdr_t = max(hdr_t, os.path.getmtime(os.path.join(CSRC, "torch_args.h")))
    bindings = []  # source, object, module, whether to compile
    for name, so in (("kv4_torch", BINDING), ("kv16_torch", BINDING16)) if torch else ():
        bsrc, bobj = os.path.join(CSRC, name + ".cpp"), os.path.join(BUILD, name + ".o")
        stale = force or not os.path.exists(bobj) or os.path.getmtime(bobj) < max(os.path.getmtime(bsrc), binding_hdr_t)
        bindings.append((bsrc, bobj, so, stale))

    def cc_binding(bsrc, bobj):
        t = os.path.join(torch, "include")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w", "-c", bsrc, "-o", bobj, "-I", t,
               "-I", os.path.join(t, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
               "-I", cuda_include(), "-I", os.path.join(ROOT, "include")]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            raise RuntimeError(f"g++ failed for {bsrc}:\n{r.stderr}")

    with cf.ThreadPoolExecutor(max(1, min(len(jobs) + 2, os.cpu_count() or 1))) as ex:
        others = [ex.submit(cc_binding, bsrc, bobj) for bsrc, bobj, _, stale in bindings if stale]
        logs = list(ex.map(cc, jobs))
    if verbose:
        for log in logs:
            print(log)
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if jobs or not os.path.exists(LIB):
        tmp = LIB + f".{os.getpid()}.tmp"
        subprocess.check_call([nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    for other in others:
        other.result()
    for _, bobj, so, stale in bindings:
        if not stale and os.path.exists(so):
            continue
        lib = os.path.join(torch, "lib")
        tmp = so + f".{os.getpid()}.tmp"
        subprocess.check_call(["g++", "-shared", "-o", tmp, bobj, "-L", HERE, "-llookahead", "-Wl,-rpath,$ORIGIN",
                               "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"])
        os.replace(tmp, so)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
