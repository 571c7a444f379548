"""A row belongs to whole waves, so the addresses its loads take are the same for a wave's lanes, and the compiler has
to know that: the row kernels, whose loops are all unrolled, must hold no loop over the lanes' addresses. Compiled only,
no GPU."""
import os
import re
import subprocess

from mxfp4_block_scaled_02_amd import build


def test_row_kernels_hold_no_loop(tmp_path):
    out = tmp_path / "int8_quant.s"
    r = subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, "int8_quant.hip"),
                        "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    kernels = re.findall(r"^(\S*\d+row_kernelI\S*):(.*?)^\.Lfunc_end", out.read_text(), re.M | re.S)
    assert len(kernels) == 63  # three types, three modes, seven sizes
    looping = []
    for name, body in kernels:
        seen = set()
        for line in body.splitlines():
            if label := re.match(r"(\.L\w+):", line):
                seen.add(label[1])
            elif (branch := re.match(r"\s+s_c?branch\w*\s+(\.L\w+)", line)) and branch[1] in seen:
                looping.append(name)
    assert not looping, sorted(set(looping))
