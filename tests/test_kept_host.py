"""What the library keeps of the driver's answers, on the CPU: the header compiled with the host
compiler. A query that failed is asked again; one that was answered is not."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "w4a8_ptq_linear_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "kept.h"
int main() {
  oq::Kept<int, int> kept;
  int asked = 0, v = -1;
  auto fails = [&](int* x) { ++asked; *x = 3; return false; };
  auto gives = [&](int* x) { ++asked; *x = 7; return true; };
  bool ok = !kept.get(1, &v, fails) && v == 3;      // this call's alone
  ok = ok && !kept.get(1, &v, fails) && asked == 2; // asked again
  ok = ok && kept.get(1, &v, gives) && v == 7 && asked == 3;
  ok = ok && kept.get(1, &v, fails) && v == 7 && asked == 3;   // kept
  ok = ok && !kept.get(2, &v, fails) && asked == 4; // another key
  std::vector<std::thread> ts;
  int got[8] = {};
  for (int i = 0; i < 8; ++i)
    ts.emplace_back([&, i] {
      for (int n = 0; n < 1000; ++n) kept.get(10 + n, &got[i], [n](int* x) { *x = n; return n % 3 != 0; });
    });
  for (auto& t : ts) t.join();
  for (int g : got) ok = ok && g == 999;
  std::puts(ok ? "ok" : "wrong");
}
"""


def test_a_failed_query_is_asked_again(tmp_path):
    src, exe = tmp_path / "k.cpp", str(tmp_path / "k")
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", exe], check=True)
    assert subprocess.run([exe], check=True, capture_output=True, text=True).stdout == "ok\n"
