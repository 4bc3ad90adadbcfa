"""Compile libdtree.so (sm_100a) in-tree with nvcc.

    python draft_tree_construction_markov_b200/build.py [--verbose]

The shared library lands next to this file so that it travels with the
repository; nothing is installed into site-packages.
"""
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdtree.so")
SOURCES = ["api_build.cu", "markov_gemm.cu", "frontier.cu", "accept.cu", "verify_attn.cu",
           "treeflash.cu", "attn_tc.cu", "accept_noalloc.cu", "load_policy.cu", "pbuild.cu",
           "calibration.cu", "kv_cache.cu", "paged_attn.cu", "paged_tc.cu", "paged_decode.cu",
           "logits.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "--shared", "-Xcompiler", "-fPIC",
    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
    "--expt-relaxed-constexpr", "--threads", "0",
]


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "dtree.h")]
    return any(os.path.getmtime(d) > t for d in deps)


# Registers a thread has at launch in the paged attention's tile kernels whose warps deal them out
# anew (TcShape::kLaunchRegs), by the type of the cache and the row tiles of a block.
LAUNCH_REGS = {(1, 2): 168, (2, 1): 80, (3, 1): 80, (2, 2): 128, (3, 2): 128}


def check_registers(log):
    """Raises where the compiler (its -v output) gave such a kernel another number than its shares are
    made for: the library would refuse to launch it, and its calls would fail."""
    for d, code, tiles, regs in re.findall(
            r"Compiling entry function '\S*paged_tc_kernelILi(\d+)ELi(\d)ELi(\d)E(?:(?!Compiling entry).)*?"
            r"Used (\d+) registers", log, re.S):
        want = LAUNCH_REGS.get((int(code), int(tiles)))
        if want and int(regs) != want:
            raise RuntimeError(f"paged_tc_kernel<{d}, {code}, {tiles}> has {regs} registers a thread, not {want}: "
                               "this compiler needs other shares in TcShape (csrc/paged_tc.cu)")


def build(force=False, verbose=False):
    if not force and not _stale():
        return LIB
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    cmd = [NVCC, *FLAGS, "-Xptxas", "-v", "-o", LIB + ".tmp", *srcs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 or verbose:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed building libdtree.so")
    check_registers(r.stdout + r.stderr)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
