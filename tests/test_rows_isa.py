"""Spills of the row kernels (norms, 8-bit rows), on the generated gfx950 assembly: none
but where a lane holds more float32 values than its registers do."""
import os
import re
import subprocess

import pytest

from post_weight_quantization_26_amd import build_lib
from test_asm_mfma_isa import _hipcc

# the gradient of float32 rows above 8192 columns, quantised rows above 32768
KNOWN = ("norm_back_kernelILi0ELi16ELi4E", "quantize_rows8_kernelILi0ELi16ELi8E",
         "quantize_rows8_kernelILi1ELi16ELi8E", "quantize_rows8_kernelILi2ELi16ELi8E")


@pytest.mark.parametrize("src,least", [("norm.hip", 30), ("rows8.hip", 15)])
def test_row_kernels_spill_nothing(tmp_path, src, least):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc is not available")
    out = str(tmp_path / "rows.s")
    res = subprocess.run([cc, *build_lib.COMMON, "--cuda-device-only", "-S",
                          os.path.join(build_lib.CSRC, src), "-o", out],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    found = re.findall(r"\.name:\s+(\S+kernel\S+)\n(?:.*\n)*?\s+\.vgpr_spill_count:\s+(\d+)",
                       open(out).read())
    assert len(found) >= least
    spilled = [(name, n) for name, n in found
               if int(n) and not any(k in name for k in KNOWN)]
    assert not spilled
