"""Wait states between the FP16 matrix instructions of the orthogonalisation's
products, whose results lie in ordinary VGPRs, and the first vector or memory
instruction that reads them: at least 11 (an 8-pass instruction) on every path
of the built gfx950 code, walked as for the layer's own products."""

import os
import re
import shutil
import subprocess

import pytest

from tests.test_mfma_hazards import LIB, LLVM, REQUIRED, distances

BUNDLE = b"__CLANG_OFFLOAD_BUNDLE__"


@pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")
@pytest.mark.skipif(not shutil.which(os.path.join(LLVM, "llvm-objdump")), reason="llvm-objdump missing")
def test_fp16_mfma_results_read_after_enough_wait_states(tmp_path):
    fat = tmp_path / "fat.bin"
    subprocess.run([os.path.join(LLVM, "llvm-objcopy"), "--dump-section=.hip_fatbin=" + str(fat), LIB,
                    str(tmp_path / "discard.so")], check=True)
    data = fat.read_bytes()
    starts = [m.start() for m in re.finditer(BUNDLE, data)] + [len(data)]        # one bundle per source
    read = []
    for i, (a, b) in enumerate(zip(starts, starts[1:])):
        one, co = tmp_path / f"b{i}.bin", tmp_path / f"k{i}.co"
        one.write_bytes(data[a:b])
        subprocess.run([os.path.join(LLVM, "clang-offload-bundler"), "--unbundle", "--type=o", "--input=" + str(one),
                        "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", "--output=" + str(co)], check=True)
        listing = subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", "--mcpu=gfx950", str(co)], check=True,
                                 capture_output=True, text=True).stdout
        read += [r for r in distances(listing, "v_mfma_f32_16x16x32_f16", 30) if r[2] is not None]
    kernels = {f for _, f, _ in read}
    assert any("k_orth_gemm" in f for f in kernels), "no FP16 result read found: the checker sees nothing"
    short = [r for r in read if r[2] < REQUIRED]
    assert not short, f"VGPR results read too early: {short[:5]}"
