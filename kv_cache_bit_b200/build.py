"""Build libkvq.so (CUDA, sm_100a) into kv_cache_bit_b200/_lib/.

nvcc cross-compiles without a GPU.  The library has two translation units:
csrc/kvq_api.cu (the block cache) and csrc/kvq_pages.cu (the paged cache),
each of which includes its kernel headers.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libkvq.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

# translation unit -> the headers of csrc/ that only it includes
UNITS = {"kvq_api.cu": ("kvq_decode_mma.cuh", "kvq_decode_simple.cuh", "kvq_quant.cuh", "kvq_quant_rows.cuh"),
         "kvq_pages.cu": ("kvq_pages.cuh", "kvq_pages_attn.cuh", "kvq_pages_step.cuh", "kvq_pages_tile.cuh")}


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


TEST_LIB = os.path.join(OUT_DIR, "libkvq_waittest.so")

# Not --split-compile: it halves the time, but takes registers and spills by chance, so that one source gave the
# 8192-token prompt of the paged attention 1040 or 1165 us from build to build (1002 without it).
_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
          "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]


def _deps(unit):
    others = {h for u, hs in UNITS.items() if u != unit for h in (u, *hs)}
    return [p for p in sources() if os.path.basename(p) not in others] + [os.path.join(ROOT, "include", "kvq.h"),
                                                                           __file__]


def _stale(out, deps):
    return not os.path.exists(out) or os.path.getmtime(out) < max(os.path.getmtime(p) for p in deps)


def build(force: bool = False, verbose: bool = False, test_lib: bool = True) -> str:
    """Build libkvq.so and, unless test_lib is False, the test build
    libkvq_waittest.so (the same sources with KVQ_WAIT_TEST: the kernels'
    main-loop waits can be made to give up at once, for the failure-path
    test).  The units compile in parallel."""
    os.makedirs(OUT_DIR, exist_ok=True)
    targets = [(LIB, ())] + ([(TEST_LIB, ("-DKVQ_WAIT_TEST",))] if test_lib else [])
    jobs, links = [], []
    for out, extra in targets:
        objs = []
        for unit in UNITS:
            obj = out[:-len(".so")] + "." + unit[:-len(".cu")] + ".o"
            objs.append(obj)
            if force or _stale(obj, _deps(unit)):
                cmd = [NVCC, *_FLAGS, *(["-Xptxas=-v"] if verbose else []), *extra, "-c", "-o", obj + ".tmp",
                       os.path.join(CSRC, unit)]
                jobs.append((obj, subprocess.Popen(cmd)))
        links.append((out, objs))
    for obj, proc in jobs:
        if proc.wait() != 0:
            raise subprocess.CalledProcessError(proc.returncode, "nvcc " + obj)
        os.replace(obj + ".tmp", obj)
    for out, objs in links:
        if force or _stale(out, objs):
            subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", out + ".tmp", *objs],
                           check=True)
            os.replace(out + ".tmp", out)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
