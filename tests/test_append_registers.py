"""Registers of the norm, rotation and append, as ptxas reports them (CPU): five CTAs of 128 threads to an SM for every
instance whose steps are full, and nothing to speak of spilled."""
import os
import re
import shutil
import subprocess

import pytest

from nvfp4_paged_kv_02_gb300 import _build


@pytest.mark.slow
def test_five_ctas_where_steps_are_full(tmp_path):
    r = subprocess.run([_build.nvcc(), *_build.NVCC_FLAGS, "-Xptxas", "-v", "-c", os.path.join(_build.CSRC, "norm_rope.cu"),
                        "-o", str(tmp_path / "norm_rope.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    if not shutil.which("c++filt"):
        pytest.skip("needs c++filt")
    text = subprocess.run(["c++filt"], input=r.stderr, capture_output=True, text=True).stdout
    found = re.findall(r"norm_rope_append_kernel<(\w+), (\d), (\w+), (\w+)>.*?(\d+) bytes spill stores.*?Used (\d+) registers",
                       text, re.S)
    found = {x[:4]: (int(x[4]), int(x[5])) for x in found}
    assert len(found) == 40
    for (bf16, mode, mixed, axes), (spilled, registers) in found.items():
        what = (bf16, mode, mixed, axes, registers, spilled)
        assert spilled <= 4, what
        if mixed == "false" or axes == "true" or mode == "0":
            assert -(-registers // 8) * 8 * 128 * 5 <= 65536, what
