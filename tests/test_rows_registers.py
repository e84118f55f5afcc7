"""The row kernels hold a row in registers: none of them uses scratch memory, as the compiler reports it."""
import os
import re
import subprocess

import pytest

from structured_rank_matmul_amd import build


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
def test_no_row_kernel_uses_scratch(tmp_path):
    r = subprocess.run([build.HIPCC, *build.HIP_FLAGS, "--cuda-device-only", "-Rpass-analysis=kernel-resource-usage", "-c",
                        os.path.join(build.CSRC, "rows.hip"), "-o", str(tmp_path / "rows.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    names = re.findall(r"Function Name: (\S+)", r.stderr)
    scratch = [int(v) for v in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", r.stderr)]
    assert len(names) == len(scratch) and sum("rows_kernel" in n for n in names) == 3 * (10 + 11)
    assert not any(scratch), [(n, s) for n, s in zip(names, scratch) if s]
