"""The rules of the waits in the kernels on the CTA-wide tensor instructions, on the host: a wait ends, says whether what it
waited for is there, and is heard of."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_command_execution_gb300", "csrc")

HOST = r"""
#include <cassert>
#include <initializer_list>
#include "cache_wait.cuh"
using namespace cmdx;

int main() {
  uint64_t clock = 5, step = 1;
  uint32_t tries = 0, looks = 0, yes_at = 0;
  const auto ready = [&] { return ++tries == yes_at; };
  const auto now = [&] { ++looks; return clock += step; };
  volatile uint32_t stop = 0;
  // what comes is waited for, and the word stays as it was
  for (uint32_t at : {1u, 2u, 255u, 256u, 257u, 100000u}) {
    tries = 0;
    yes_at = at;
    assert(wait_until(&stop, ready, now) && tries == at && stop == 0);
  }
  assert(looks <= 100000 / 256 + 6);
  // what never comes is given up after the time that it has, not before, and the word is set
  for (uint64_t s : {kPatience / 100, kPatience / 2, 2 * kPatience}) {
    tries = looks = yes_at = 0;
    stop = 0;
    step = s;
    const uint64_t began = clock;
    assert(!wait_until(&stop, ready, now) && stop == 1);
    assert(clock - began > kPatience && clock - began <= kPatience + 2 * s + 1);
  }
  // once the word is set, a wait ends soon, without the clock; unless what it waits for is there
  tries = looks = yes_at = 0;
  assert(!wait_until(&stop, ready, now) && tries <= 256 && looks == 0 && stop == 1);
  tries = 0;
  yes_at = 3;
  assert(wait_until(&stop, ready, now) && tries == 3);
  // what is on its way is waited for whatever the word says
  tries = looks = 0;
  yes_at = 5000;
  step = 1;
  assert(wait_anyway(&stop, ready, now) && tries == 5000 && stop == 1);
  stop = 0;
  tries = 0;
  assert(wait_anyway(&stop, ready, now) && stop == 0);
  tries = yes_at = 0;
  step = kPatience / 2;
  assert(!wait_anyway(&stop, ready, now) && stop == 1);
  return 0;
}
"""


def test_waits(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    (tmp_path / "w.cpp").write_text(HOST)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(tmp_path / "w.cpp"), "-o", str(tmp_path / "w")], check=True)
    subprocess.run([str(tmp_path / "w")], check=True, timeout=60)


@pytest.mark.parametrize("name", ["cache_drafts_tc.cu", "cache_weigh_tc.cu"])
def test_what_a_wait_says_is_heeded(name):
    """Who copies by TMA stops when a wait has given up, what a CTA has on its way (copies, products) is waited for before it
    ends, and results are written as such only where the word is clear after the last wait."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert re.search(r"if \(!(?:\(going = )?warp_wait\(s\.stop, smem_u32\(&s\.empty\[", text)
    assert re.search(r"wait_own\(s\.stop, smem_u32\(&s\.full\[", text)
    assert re.search(r"tcgen05_commit\(one, smem_u32\(&s\.end\)\);\s*wait_own\(s\.stop, smem_u32\(&s\.end\), 0\);", text)
    if name == "cache_weigh_tc.cu":
        before, after = text.split("if (gave_up(s.stop)) {")
        assert "weights[t] = " not in before and re.match(r"\s*if \(t >= g\.lo && t < g\.n\) weights\[t\] = CUDART_NAN_F;\s*\} else if", after)
        assert "wait(s.stop" not in after[:after.index("template <class T, int DP>")]
    else:
        assert re.search(r"if \(any\) wait\(s\.stop, smem_u32\(&s\.done\[w\]\), \(count - 1\) & 1\);\s*tcgen05_after_sync\(\);\s*"
                         r"if \(gave_up\(s\.stop\)\) l = CUDART_NAN_F;", text)
        assert re.search(r"__all_sync\(~0u, bad && !gave_up\(s\.stop\)\)\) \{\s*add_infinite", text)
