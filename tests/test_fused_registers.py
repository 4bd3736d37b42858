"""The register counts that the chunked fused products rest on (CPU only: the compiler's report)."""

import os
import re
import subprocess

from blas3_tensor_core_gb300 import build


def test_chunked_copies_get_the_registers_that_their_warps_share_out(tmp_path):
    """setmaxnreg moves registers between the warps of a block; what it hands the epilogue has to be
    there from the launch on. The six copies that use it (three tiles, forward and backward) must
    have FUSED_LAUNCH_REGS of them."""
    with open(os.path.join(build.CSRC, "bm_fused_kernel.cuh")) as f:
        launch = int(re.search(r"FUSED_LAUNCH_REGS = (\d+)", f.read()).group(1))
    cmd = [build.nvcc(), *build.NVCC_FLAGS, "-Xptxas", "-v", "-I", build.INCLUDE, "-I", build.CSRC, "-c",
           os.path.join(build.CSRC, "bm_fused.cu"), "-o", str(tmp_path / "fused.o")]
    report = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    counts, name = {}, None
    for line in report.splitlines():
        if (m := re.search(r"Compiling entry function '(\S+)'", line)) is not None:
            name = m.group(1)
        elif (m := re.search(r"Used (\d+) registers", line)) is not None and name is not None:
            counts[name] = int(m.group(1))
    chunked = {k: v for k, v in counts.items() if re.search(r"bm_gemm_fused_kernelI\w+ELb[01]ELb1EE", k)}
    assert len(chunked) == 6, sorted(counts)
    assert all(v >= launch for v in chunked.values()), chunked
