"""Build libbf16opt.so (the C-ABI library) for gfx950 with hipcc, in-tree: the
sources side by side into a temporary folder, then linked.

Floating-point flags: -ffp-contract=off (no implicit multiply-add fusion: the
update's op sequence is fixed), correctly rounded fp32 divide/sqrt and fp32
denormals kept (HIP's defaults, stated explicitly), and packed-fp32
instructions disabled.
"""
from concurrent.futures import ThreadPoolExecutor
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libbf16opt.so")
SOURCES = [os.path.join(CSRC, "bfo_kernels.hip"), os.path.join(CSRC, "bfo_abi.cpp"),
           os.path.join(CSRC, "bfo_control.cpp"), os.path.join(CSRC, "bfo_checkpoint.cpp"),
           os.path.join(CSRC, "bfo_layernorm.hip"), os.path.join(CSRC, "bfo_logits.hip"),
           os.path.join(CSRC, "bfo_ops.cpp"), os.path.join(CSRC, "bfo_rmsnorm.hip"),
           os.path.join(CSRC, "bfo_activation.hip"), os.path.join(CSRC, "bfo_rotary.hip"),
           os.path.join(CSRC, "bfo_block.cpp")]
ARCH = os.environ.get("BFO_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-pthread",
    "-ffp-contract=off",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def hipcc():
    return os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)


def build(verbose: bool = False, extra=()) -> str:
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as folder:
        objects = [os.path.join(folder, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(lambda so: _run([hipcc(), *HIPCC_FLAGS, *extra, "-c", "-o", so[1], so[0]], verbose),
                          zip(SOURCES, objects)))
        _run([hipcc(), *HIPCC_FLAGS, *extra, "-shared", "-o", tmp, *objects], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
