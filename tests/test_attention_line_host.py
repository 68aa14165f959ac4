"""How the attention's line of units is cut, on the host: the header's own function, compiled into a
small program (nvcc, no GPU)."""
import subprocess

import pytest

from diffusion_decoding_gb300 import build as cuda_build

PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "attention_line.cuh"
int main(int argc, char** argv) {
  for (int i = 1; i + 1 < argc; i += 2)
    std::printf("%d ", dllm::unit_log2_of(std::atoll(argv[i]), std::atoi(argv[i + 1]), 6));
}
"""


@pytest.fixture(scope="module")
def unit_log2(tmp_path_factory):
    d = tmp_path_factory.mktemp("line")
    (d / "line.cu").write_text(PROGRAM)
    subprocess.run([cuda_build.nvcc(), *cuda_build.ARCH, "-std=c++17", "-I", cuda_build.INCLUDE, "-I",
                    cuda_build.CSRC, "-o", str(d / "line"), str(d / "line.cu")], check=True)

    def call(pairs):
        args = [str(x) for p in pairs for x in p]
        return [int(x) for x in subprocess.run([str(d / "line"), *args], check=True, capture_output=True,
                                               text=True).stdout.split()]
    return call


def test_units_fit_the_line(unit_log2):
    # segments up to 2^30 (B * n * heads), lengths up to 2^30: fewer than 2^31 units, each of at most
    # 2^30 entries (the kernels add lengths and units in 32 bits)
    pairs = [(s, n) for a in (0, 3, 20, 27, 29, 30) for s in (1 << a, (1 << a) - 1) if s
             for b in (0, 6, 9, 17, 29, 30) for n in (0, (1 << b) - 1, 1 << b)]
    units = lambda s, n, lg: s * max(1, -(-n >> lg))  # noqa: E731
    for (s, n), lg in zip(pairs, unit_log2(pairs)):
        assert 6 <= lg <= 30, (s, n, lg)
        assert units(s, n, lg) < 1 << 31, (s, n, lg)
