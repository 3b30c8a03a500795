"""Set-up that the first call on each device does (csrc/per_device.h), compiled
by the host compiler and run with two made-up devices; and that no kernel's
set-up is kept once a process, read from the sources."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "backward_tcgen05_tma_gemms_gb300", "csrc")

PROGRAM = r"""
#include <cassert>
#include <thread>
#include "per_device.h"
int main() {
  tps::PerDevice<int> known;
  int made[3] = {0, 0, 0}, value = -1;
  auto on = [&](int device, bool able) {
    return known.get(device, &value, [&](int* v) { ++made[device]; *v = 10 * device + 7; return able; });
  };
  assert(on(1, true) && value == 17);
  assert(on(0, true) && value == 7);                       // its own set-up, although another device had one
  assert(on(1, true) && value == 17 && on(0, true) && value == 7);
  assert(made[0] == 1 && made[1] == 1);
  value = -1;
  assert(!on(2, false) && value == -1 && made[2] == 1);    // what failed is not kept ...
  assert(on(2, true) && value == 27 && made[2] == 2);      // ... but asked for again
  assert(!on(-1, true));
  int calls = 0;
  tps::PerDevice<int> shared;
  auto many = [&] {
    for (int i = 0; i < 1000; ++i) {
      int v = 0;
      assert(shared.get(i % 5, &v, [&](int* w) { ++calls; *w = i % 5; return true; }) && v == i % 5);
    }
  };
  std::thread a(many), b(many);
  a.join();
  b.join();
  assert(calls == 5);
  return 0;
}
"""


def test_first_call_on_each_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    subprocess.run([str(exe)], check=True, timeout=60)


def test_no_set_up_once_a_process():
    for f in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        for m in re.finditer(r"call_once\(", text):  # the driver's entry point is no device's
            assert "cudaGetDriverEntryPoint" in text[m.end():m.end() + 300], f
