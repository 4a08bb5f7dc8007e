"""The 8-bit product's warpgroups share out the registers that its blocks launch with;
the launch refuses a kernel that was given fewer.  This compiler gives it as many."""
import re
import subprocess
from pathlib import Path

SOURCE = Path(__file__).parent.parent / "qwen3_dense_decoder_gb300" / "csrc" / "k_i8_matmul.cu"


def test_the_kernels_launch_with_the_registers_that_they_share_out(tmp_path):
    from qwen3_dense_decoder_gb300 import buildlib
    r = subprocess.run([buildlib.nvcc(), *buildlib.ARCH, *buildlib.FLAGS, "-Xptxas", "-v", "-c", str(SOURCE), "-o", str(tmp_path / "k.o")],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    want = int(re.search(r"R_LAUNCH = (\d+)", SOURCE.read_text()).group(1))
    used = re.findall(r"Compiling entry function '\S*i8_gemm_kernel\S*'.*?Used (\d+) registers", r.stdout + r.stderr, re.S)
    assert len(used) == 2 and all(int(u) >= want for u in used), used
