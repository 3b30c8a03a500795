"""What the shard-aware fp32 kernel (gemm_simt.cu) does not compute, it refuses:
a host program asks the built library for it, with 2^23 rows, which are more
than its grid takes, so that a form that it does know is refused for that and
nothing is launched either way."""
import subprocess

from backward_tcgen05_tma_gemms_gb300 import build
from test_abi_host import lib  # noqa: F401  (fixture)

PROGRAM = r"""
#include <cstdio>
#include "internal.cuh"
int main() {
  for (int mode : {tps::EPI_STORE, tps::EPI_ACT_FWD, tps::EPI_GLU_FWD, tps::EPI_CE_STATS, tps::EPI_CE_LSE, tps::EPI_CE_GRAD,
                   tps::EPI_LINEAR}) {
    tps::GemmDesc g;
    g.M = 1 << 23; g.N = 1; g.K = 1;
    g.epi.mode = static_cast<decltype(g.epi.mode)>(mode);
    printf("%d ", tps::launch_gemm_simt(g, nullptr, nullptr));
  }
}
"""


def test_refused_forms(lib, tmp_path):  # noqa: F811
    src, exe = tmp_path / "t.cu", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, str(src), "-o", str(exe),
                    build.LIB, "-Xlinker", f"-rpath={build.PKG}"], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=120).stdout.split()
    shape, arg = "1", "9"
    assert out == [shape, shape, arg, arg, arg, arg, arg]
