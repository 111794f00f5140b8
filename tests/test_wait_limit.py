"""The limit of the prompt kernels' waits (csrc/wait_limit.h), compiled for the host: it counts the time in which the
block looks, not that in which its process is off the GPU."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_kv_gb300", "csrc")
MAIN = r"""
#include <stdio.h>
#include <stdlib.h>
#include "wait_limit.h"
// looks `gap` ns apart, `looks` of them, the one in the middle `jump` ns later: how many until the limit is over
int main(int argc, char** argv) {
  const uint64_t gap = strtoull(argv[1], 0, 10), looks = strtoull(argv[2], 0, 10), jump = strtoull(argv[3], 0, 10);
  uint64_t now = 4200000000ull;  // the lower half wraps soon
  paris::WaitLimit limit((uint32_t)now);
  for (uint64_t i = 1; i <= looks; ++i) {
    now += gap + (i == looks / 2 ? jump : 0);
    if (limit.over((uint32_t)now)) {
      printf("%llu", (unsigned long long)i);
      return 0;
    }
  }
  printf("0");
  return 0;
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    d = tmp_path_factory.mktemp("wait")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(d / "main.cpp"), "-o", str(d / "main")], check=True)
    return lambda *a: int(subprocess.run([str(d / "main"), *map(str, a)], check=True, capture_output=True).stdout)


def test_a_wait_ends_after_four_seconds_of_looking(run):
    assert run(1000, 5000000, 0) == 4000001
    assert run(1000, 3999999, 0) == 0
    assert run(1000000, 5000, 0) == 4001


def test_time_off_the_gpu_does_not_end_it(run):
    assert run(1000, 1000000, 10 ** 10) == 0       # ten seconds away, one second of looking
    assert run(1000, 5000000, 10 ** 10) < 4000001  # still over after four seconds of looking
    assert run(1000, 5000000, 10 ** 10) > 3970000


def test_it_ends_also_where_every_look_is_late(run):
    assert run(10 ** 9, 1000, 0) == 201
    assert run(2 * 10 ** 7, 1000, 0) == 201
