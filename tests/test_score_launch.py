"""Launch rules of the score-rule and paged kernels (host code of cp_score.h),
compiled into a small program that touches no device."""
import os
import subprocess

import pytest

from context_attention_dits_gb300 import build

PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "cp_score.h"
int main(int argc, char** argv) {
  const int sms = std::atoi(argv[1]);
  std::printf("%d %d %d %d\\n", cp::cluster_for(1.5, 76, 64, 0, 0, 1.0, true, sms),
              cp::paged_grid(128, true, 100000, sms), cp::paged_grid(128, false, 100000, sms),
              cp::paged_grid(64, true, 5, sms));
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("launch")
    (d / "rules.cu").write_text(PROGRAM)
    exe = d / "rules"
    subprocess.run([build.nvcc_path(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-o", str(exe),
                    str(d / "rules.cu")], check=True)
    return str(exe)


# 76 items of 64 tiles: clusters of two where as many multiprocessors again would idle; decode: one wave of CTAs,
# at most the 304 that the workspace has room for
@pytest.mark.parametrize("sms,want", [(152, [2, 304, 152, 5]), (76, [1, 152, 76, 5]), (160, [2, 304, 152, 5]),
                                      (2, [1, 4, 2, 4])])
def test_rules_follow_the_device(program, sms, want):
    got = subprocess.run([program, str(sms)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == want
