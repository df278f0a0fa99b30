"""What the compiler reports of the kernels around verification: tiles and vectors
that are meant to stay in registers do, no kernel has scratch memory."""
import os
import re
import subprocess

import pytest

from speculative_decoding_verification_pipeline_amd import build


@pytest.mark.parametrize("source,kernels", [("ss_cache.hip", 16), ("ss_probs.hip", 6)])
def test_no_kernel_has_scratch(source, kernels, tmp_path):
    cmd = [build.hipcc(), *build.CFLAGS, "-I", build.INCLUDE, "-x", "hip", "--cuda-device-only", "-c",
           os.path.join(build.CSRC, source), "-o", str(tmp_path / "k.o"),
           "-Rpass-analysis=kernel-resource-usage"]
    out = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    names = re.findall(r"Function Name: (\S+)", out)
    scratch = [int(n) for n in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", out)]
    assert len(names) == len(scratch) >= kernels
    assert not [(n, s) for n, s in zip(names, scratch) if s]
