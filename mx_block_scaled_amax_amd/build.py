"""Build libqf8.so (the HIP kernels and the C ABI of include/qf8.h) for gfx950 with hipcc."""
import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libqf8.so")
SOURCES = ["qf8_api.cpp", "qf8_tensor.hip", "qf8_block.hip", "qf8_mx.hip", "qf8_dequant.hip", "qf8_requant.hip", "qf8_fp4.hip",
           "qf8_experts.hip", "qf8_norm.hip", "qf8_gate.hip", "qf8_layer.hip", "qf8_clip.hip", "qf8_matmul.hip",
           "qf8_matmul_e4m3_e4m3.hip", "qf8_matmul_e4m3_e5m2.hip", "qf8_matmul_e5m2_e4m3.hip", "qf8_matmul_e5m2_e5m2.hip"]
ARCH = "gfx950"


def hipcc():
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found: the qf8 library is built with ROCm's hipcc for gfx950")


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + " ".join(cmd) + "\n" + err)
    return err


def build(verbose=False):
    """Compile every source (a few at a time) and link libqf8.so; always recompiles."""
    tmp = LIB + ".tmp"
    flags = [hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
             "-Wall", "-Wno-unused-command-line-argument",
             # packed fp32 VALU ops are kept out of the generated code
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", os.path.join(ROOT, "include")]
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, os.path.splitext(s)[0] + ".o") for s in SOURCES]
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as ex:
            errs = list(ex.map(lambda so: _run(flags + ["-c", os.path.join(CSRC, so[0]), "-o", so[1]]),
                               zip(SOURCES, objs)))
        errs.append(_run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-o", tmp] + objs))
    err = "\n".join(e for e in errs if e.strip())
    if verbose and err:
        print(err, file=sys.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
