"""Host logic of the launch code: what the runtime answers is kept, a failed question is not."""
import os
import shutil
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_vector_append_b200", "csrc")

PROGRAM = r"""
#include "tq_memo.cuh"
#include <cstdio>

int main() {
  static tq::Memo<3> memo;
  int asked = 0, got = -1;
  auto ask = [&](int* a) {                    // fails the first time, then answers 4 + times asked
    *a = 4 + asked;
    return ++asked > 1;
  };
  if (memo.get(1, ask, &got) || got != -1) return 1;       // no answer, and none made up
  if (!memo.get(1, ask, &got) || got != 5) return 2;       // asked again
  if (!memo.get(1, ask, &got) || got != 5 || asked != 2) return 3;   // kept
  if (!memo.get(0, ask, &got) || got != 6) return 4;       // of its key only
  if (!memo.get(1, ask, &got) || got != 5 || asked != 3) return 5;
  int zero = -1, times = 0;
  auto none = [&](int* a) { ++times; *a = 0; return true; };
  for (int i = 0; i < 2; ++i)
    if (!memo.get(2, none, &zero) || zero != 0 || times != 1) return 6;   // 0 is an answer
  return 0;
}
"""


def test_an_answer_is_kept_and_a_failure_is_not(tmp_path):
    src, exe = tmp_path / "memo.cpp", tmp_path / "memo"
    src.write_text(PROGRAM)
    cxx = shutil.which("g++") or "g++"
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_launches_keep_no_answer_of_their_own():
    """Function-local static results would keep a failure for the life of the process."""
    for name in ("tq_attend_launch.cuh", "tq_pages.cu", "tq_pages_launch.cuh"):
        text = open(os.path.join(CSRC, name)).read()
        statics = [line.strip() for line in text.splitlines() if line.strip().startswith("static ")]
        assert all(s.startswith("static Memo<") for s in statics), (name, statics)
