"""The check that stands between the sort's counts, which lie in a workspace, and
its stores."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp4_quantized_prep_amd", "csrc")

PROGRAM = """
#include <climits>
#include "iqp_internal.h"
using iqp::is_place;
int main() {
  for (int64_t R : {(int64_t)0, (int64_t)1, (int64_t)37056, (int64_t)INT_MAX})
    for (int64_t to : {(int64_t)INT_MIN, (int64_t)INT_MIN + 1, (int64_t)-1065353216, (int64_t)-2, (int64_t)-1, (int64_t)0, (int64_t)1, R - 1, R,
                       (int64_t)1065353216, (int64_t)INT_MAX})
      if (is_place((int32_t)to, R) != (to >= 0 && to < R)) return 1;
  return 0;
}
"""


def test_places_outside_the_batch_are_none(tmp_path):
    """Whatever bits a count holds, a float's of either sign among them."""
    (tmp_path / "a.cpp").write_text(PROGRAM)
    cmd = ["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__=1", "-I" + CSRC, "-I/opt/rocm/include", "a.cpp", "-o", "a"]
    r = subprocess.run(cmd, cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(tmp_path / "a")]).returncode == 0


def test_places_are_checked_before_they_are_stored():
    """The sort's only store to a place that it looked up."""
    with open(os.path.join(CSRC, "moe_route.hip")) as f:
        text = f.read()
    assert re.findall(r"(?:(if \(.*?\)) )?p\.rows\[to\] =", text) == ["if (is_place(to, p.R))"]
    assert "p.slots[i] = to;" in text and "else to = -1;" in text
