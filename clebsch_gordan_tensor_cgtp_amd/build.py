"""Build libcgtp.so in-tree with hipcc for gfx950.

    python -m clebsch_gordan_tensor_cgtp_amd.build [--warm c1 c2 ...]

The host planner/ABI (C++) and the fixed kernels (HIP) are compiled into one
shared library next to this file, and the compiled calls of the block and
optimizer entry points (``csrc/torch``) into a Python module beside it (left out
where there is no torch).  ``--warm`` additionally creates the plans of the named
workloads so that their generated modules are compiled by hipRTC now and stored
in the on-disk cache (``jit_cache`` next to the library).
"""
import argparse
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libcgtp.so")
CALLS = os.path.join(HERE, "_calls.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

ROCM_INC = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")
GPU_FLAGS = ["--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def sources():
    csrc = os.path.join(HERE, "csrc")
    return sorted(glob.glob(os.path.join(csrc, "*.cpp"))) + sorted(glob.glob(os.path.join(csrc, "*.hip")))


def _compile(args):
    cmd, verbose = args
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    return r.returncode, r.stdout + r.stderr


def build(verbose: bool = False) -> str:
    """Host C++ sources are compiled as plain C++, the .hip sources for gfx950; then linked."""
    from concurrent.futures import ThreadPoolExecutor
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    inc = ["-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc")]
    jobs, objs = [], []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        objs.append(obj)
        if src.endswith(".hip"):
            cmd = [HIPCC, "-O2", "-std=c++17", "-fPIC", *GPU_FLAGS, *inc, "-c", src, "-o", obj]
        else:
            cmd = [HIPCC, "-O2", "-std=c++17", "-fPIC", "-x", "c++", "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INC, *inc, "-c", src,
                   "-o", obj]
        jobs.append((cmd, verbose))
    with ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
        for rc, log in ex.map(_compile, jobs):
            if rc != 0:
                sys.stderr.write(log)
                raise RuntimeError("hipcc failed building libcgtp.so")
    tmp = LIB + f".tmp{os.getpid()}"
    rc, log = _compile(([HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", *objs, "-lhiprtc", "-ldl", "-o", tmp],
                        verbose))
    if rc != 0:
        sys.stderr.write(log)
        raise RuntimeError("linking libcgtp.so failed")
    os.replace(tmp, LIB)
    build_calls(verbose)
    return LIB


def build_calls(verbose: bool = False):
    """The Python module of the block and optimizer calls (torch's headers, linked against libcgtp); None
    where there is no torch, which the library itself does not need."""
    import importlib.util
    import sysconfig
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        print("torch is not installed: libcgtp.so is built, the Python calls (_calls.so) are not", file=sys.stderr)
        return None
    torch = os.path.dirname(spec.origin)
    obj = os.path.join(HERE, "_build", "calls.cpp.o")
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], ROCM_INC, os.path.join(ROOT, "include")]
    tmp = CALLS + f".tmp{os.getpid()}"
    for cmd in ([HIPCC, "-O2", "-std=c++17", "-fPIC", "-x", "c++", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
                 *[f"-I{i}" for i in inc], "-c", os.path.join(HERE, "csrc", "torch", "calls.cpp"), "-o", obj],
                [HIPCC, "-shared", "-fPIC", obj, "-L" + HERE, "-l:libcgtp.so", "-Wl,-rpath,$ORIGIN",
                 "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip", "-o", tmp]):
        rc, log = _compile((cmd, verbose))
        if rc != 0:
            sys.stderr.write(log)
            raise RuntimeError("building _calls.so failed")
    os.replace(tmp, CALLS)
    return CALLS


def warm(names):
    """Create the named workloads' plans (both dtypes) and build the modules that are otherwise
    compiled on first use: the backward of uvw plans (batched or convolution)."""
    sys.path.insert(0, ROOT)
    from clebsch_gordan_tensor_cgtp_amd import binding, synth
    for name in names:
        for dtype in ("f32", "f64"):
            spec = {**synth.WORKLOADS, **synth.EXTRA_WORKLOADS}[name]
            plan = binding.plan_for(spec, dtype)
            if spec.mode != "uvw":
                continue
            if hasattr(spec, "n_edges"):
                plan.conv_uvw_backward_source(0)
            else:
                plan.uvw_backward_source()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--warm", nargs="*", default=[])
    ap.add_argument("-v", action="store_true")
    a = ap.parse_args()
    print(build(a.v))
    if a.warm:
        warm(a.warm)


if __name__ == "__main__":
    main()
