"""Build the HIP library in-tree with hipcc for gfx950.

    python -m moe_layer_router_amd.build

produces moe_layer_router_amd/libmoe_layer.so from csrc/kernels.hip (the
layer), csrc/training.hip (the operators around it: layer norm, the balance
loss, Newton-Schulz orthogonalisation) and csrc/peaks.hip (peak-rate
microbenchmarks).
"""

import os
import signal
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_DIR = PKG
LIB = os.path.join(LIB_DIR, "libmoe_layer.so")
SOURCES = [os.path.join(PKG, "csrc", f) for f in ("kernels.hip", "training.hip", "peaks.hip")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# Packed fp32 VALU instructions are disabled for all device code.  MFMA
# results go to ordinary VGPRs (the GEMM promotes every MFMA result with
# VALU FMAs; results in AGPRs would need a copy each).
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-mllvm", "-amdgpu-mfma-vgpr-form",
         "-I", os.path.join(ROOT, "include"), "-Wall", "-Wno-unused-function"]
LINK_FLAGS = ["--offload-arch=gfx950", "-fPIC", "-shared"]


def build(verbose: bool = False) -> str:
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objs:
        # one object per source, compiled side by side
        outs = [os.path.join(objs, os.path.basename(s) + ".o") for s in SOURCES]
        cmds = [[HIPCC, *FLAGS, "-c", s, "-o", o] for s, o in zip(SOURCES, outs)]
        procs = []
        try:
            for c in cmds:
                procs.append(subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True,
                                              start_new_session=True))
            for c, p in zip(cmds, procs):
                _finish(c, *p.communicate(), p.returncode, verbose)
        finally:
            # one failed: the others, with the compilers they started, end with it
            for p in procs:
                if p.poll() is None:
                    os.killpg(p.pid, signal.SIGKILL)
                    p.communicate()
        link = [HIPCC, *LINK_FLAGS, *outs, "-o", tmp]
        r = subprocess.run(link, capture_output=True, text=True)
        _finish(link, r.stdout, r.stderr, r.returncode, verbose)
    os.replace(tmp, LIB)
    return LIB


def _finish(cmd, out, err, rc, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    # hipcc's host pass does not know the packed-fp32 feature: drop that note
    noise = "'-packed-fp32-ops' is not a recognized feature for this target (ignoring feature)"
    err = "\n".join(l for l in err.splitlines() if noise not in l)
    if rc != 0:
        raise RuntimeError(f"hipcc failed ({rc}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


if __name__ == "__main__":
    print(build(verbose=True))
