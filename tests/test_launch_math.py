"""The launches' host arithmetic (csrc/launch_math.h), compiled by itself."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_int4_tma_gb300", "csrc")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("launch_math")
    (d / "m.cpp").write_text("""#include <cstdio>
#include <cstdlib>
#include "launch_math.h"
int main(int n, char** v) {
    if (n > 2) std::printf("%u", w4g::blocks_for(std::atoi(v[1]), std::atoi(v[2])));
    else std::printf("%d", w4g::power_of_two(std::atoi(v[1])));
}
""")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, str(d / "m.cpp"), "-o", str(d / "m")], check=True)
    return str(d / "m")


@pytest.mark.parametrize("v,want", [(1, 0), (2, 1), (3, -1), (16, 4), (24, -1), (1 << 30, 30), ((1 << 30) + 1, -1),
                                    (0x7FFF0000, -1), (0x7FFFFFFF, -1)])
def test_power_of_two(program, v, want):
    """Every size returns, those above 2^30 too."""
    got = subprocess.run([program, str(v)], capture_output=True, text=True, timeout=10, check=True).stdout
    assert int(got) == want


@pytest.mark.parametrize("n,per", [(0, 8), (1, 8), (8, 8), (9, 8), (0x7FFFFFF8, 8), (0x7FFFFFFF, 8), (0x7FFFFFFF, 4),
                                   (0x7FFFFFFF, 1)])
def test_blocks_for(program, n, per):
    got = subprocess.run([program, str(n), str(per)], capture_output=True, text=True, timeout=10, check=True).stdout
    assert int(got) == -(-n // per)
