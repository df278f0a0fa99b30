"""What the compiler reports of the kernels on 8-bit pages: what is meant to stay in
registers does, no kernel has scratch memory (a spilled value that is loaded back waits
for every load before it)."""
import os
import re
import subprocess

import pytest

from speculative_decoding_verification_pipeline_amd import build


@pytest.mark.parametrize("source,kernels", [("ss_kv8.hip", 8), ("ss_attend.hip", 20)])
def test_no_kernel_has_scratch(source, kernels, tmp_path):
    cmd = [build.hipcc(), *build.CFLAGS, "-I", build.INCLUDE, "-x", "hip", "--cuda-device-only", "-c",
           os.path.join(build.CSRC, source), "-o", str(tmp_path / "k.o"),
           "-Rpass-analysis=kernel-resource-usage"]
    out = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    names = re.findall(r"Function Name: (\S+)", out)
    scratch = [int(n) for n in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", out)]
    assert len(names) == len(scratch) >= kernels
    assert not [(n, s) for n, s in zip(names, scratch) if s]
