"""The register counts that the products with epilogues of their own rest on (CPU only: the compiler's report)."""

import os
import re
import subprocess

import pytest

from blas3_tensor_core_gb300 import build


@pytest.mark.parametrize("source, copies", [("bm_glu.cu", 6), ("bm_orth.cu", 7)])
def test_every_copy_gets_the_registers_that_its_warps_share_out(tmp_path, source, copies):
    """setmaxnreg moves registers between the warps of a block; what it hands the epilogue has to be there from the
    launch on: GLU and DGLU on three tiles each, the symmetric products on two and the step on three."""
    with open(os.path.join(build.CSRC, "bm_fused_kernel.cuh")) as f:
        launch = int(re.search(r"FUSED_LAUNCH_REGS = (\d+)", f.read()).group(1))
    cmd = [build.nvcc(), *build.NVCC_FLAGS, "-Xptxas", "-v", "-I", build.INCLUDE, "-I", build.CSRC, "-c",
           os.path.join(build.CSRC, source), "-o", str(tmp_path / "unit.o")]
    report = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    counts, name = {}, None
    for line in report.splitlines():
        if (m := re.search(r"Compiling entry function '(\S+)'", line)) is not None:
            name = m.group(1)
        elif (m := re.search(r"Used (\d+) registers", line)) is not None and name is not None:
            counts[name] = int(m.group(1))
    shared = {k: v for k, v in counts.items() if "bm_gemm_epi_kernel" in k}
    assert len(shared) == copies, sorted(counts)
    assert all(v >= launch for v in shared.values()), shared
