"""Prefix attention's kernels share their block's registers out anew, which waits
forever for more than the block was launched with: what a launch asks of a kernel as
it was built, no GPU needed."""
import os
import subprocess

from block_quantized_weight_dot_gb300 import build as lib_build

SOURCE = """
#include <stdio.h>
#include "%s"
int main() {
    for (int in8 = 0; in8 < 2; ++in8)
        for (int pp = 1; pp <= 3; pp += 2) {
            const lean::PrefixRegs r = lean::prefix_regs(in8, pp);
            printf("%%d %%d %%d %%d", in8, pp, lean::prefix_threads(in8), 128 * (2 * r.rows + r.loaders + r.mma + r.issuer));
            for (int n = 8; n <= 255; ++n) printf(" %%d", (int)lean::prefix_regs_fit(n, in8, pp));
            printf("\\n");
        }
}
"""


def test_registers_handed_out(tmp_path):
    """A kernel built with n registers a thread is launched exactly where all threads' cover what its groups take; and a
    block of as many fits the 65536 of an SM."""
    src, exe = tmp_path / "regs.cu", tmp_path / "regs"
    src.write_text(SOURCE % os.path.join(lib_build.STEP, "prefix.cuh"))
    subprocess.run([lib_build.nvcc(), "-std=c++17", "--expt-relaxed-constexpr", "-o", str(exe), str(src)] + lib_build.ARCH, check=True,
                   capture_output=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()
    assert len(lines) == 4
    for line in lines:
        in8, pp, threads, handed, *fits = map(int, line.split())
        assert threads == (640 if in8 else 512) and handed <= 65536
        for n, fit in zip(range(8, 256), fits):
            assert fit == (n * threads >= handed), (in8, pp, n)
        assert fits[(96 if in8 else 128) - 8] and not fits[(96 if in8 else 128) - 8 - 8]
    launch = open(os.path.join(lib_build.STEP, "prefix.cuh")).read()
    body = launch[launch.index("lean_status launch_prefix("):]
    body = body[:body.index("step_launch(")]
    assert "prefix_regs_there(kern, S::kIn8, PP" in body  # asked before every launch
