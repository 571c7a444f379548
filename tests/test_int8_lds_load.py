"""The load that bypasses the registers takes its LDS address in the m0 register. The compiler has to know that:
code of its own that uses m0 on both sides of such a load must find its own value there. Compiled only, no GPU."""
import os
import re
import subprocess

from mxfp4_block_scaled_02_amd import build

# The compiler's own load to LDS, load_to_lds, and the compiler's own load to the first address again.
SOURCE = """
#include "%s"
typedef __attribute__((address_space(3))) void lds_void;
extern "C" __global__ void m0_order(const uint8_t* a, int v, int other) {
  __shared__ __align__(16) uint8_t lds[4096];
  lds_void* const own = (lds_void*)(lds + 16);
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)a, (short)0, 64, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, own, 16, v, 0, 0, 0);
  load_to_lds(at + other, v, window_words(a, 1, 64, 64));
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, own, 16, v, 0, 0, 0);
}
"""


def test_a_load_to_lds_keeps_the_compilers_own_m0(tmp_path):
    src, out = tmp_path / "m0_order.hip", tmp_path / "m0_order.s"
    src.write_text(SOURCE % os.path.join(build.CSRC, "gemm_int8.hip"))
    r = subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S", str(src), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    body = re.search(r"^m0_order:(.*?)s_endpgm", out.read_text(), re.M | re.S)[1]
    written, at_load = 0, []  # writes of m0 so far, at each of the three loads
    for line in body.splitlines():
        if re.match(r"\s+s_\w+\s+m0,", line):
            written += 1
        elif re.match(r"\s+buffer_load_dwordx4 .*\blds\b", line):
            at_load.append(written)
    assert len(at_load) == 3 and 0 < at_load[0] < at_load[1] < at_load[2], body
