"""State that belongs to a device is made once for each, and a failure is not kept (csrc/per_device.h, plain C++)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "per_device.h"
#include <cstdio>
#include <thread>
#include <vector>

int main() {
  fp8q::PerDevice<int> p;
  int calls = 0, v = -1;
  auto make = [&](int value, bool ok) {
    return [&calls, value, ok](int* out) { calls++; *out = value; return ok; };
  };
  if (p.get(0, &v, make(7, false)) || calls != 1) return 1;       // a failure is reported,
  if (!p.get(0, &v, make(8, true)) || v != 8 || calls != 2) return 2;  // and tried again
  if (!p.get(0, &v, make(9, true)) || v != 8 || calls != 2) return 3;  // kept
  if (!p.get(1, &v, make(10, true)) || v != 10 || calls != 3) return 4;  // the other device's own
  if (!p.get(0, &v, make(11, true)) || v != 8 || calls != 3) return 5;
  if (!p.get(63, &v, make(12, true)) || v != 12) return 6;
  if (!p.get(64, &v, make(13, true)) || v != 13 || !p.get(64, &v, make(14, true)) || v != 14) return 7;
  if (!p.get(-1, &v, make(15, true)) || v != 15) return 8;
  static fp8q::PerDevice<int> q;
  int made = 0;
  std::vector<std::thread> t;
  for (int i = 0; i < 8; i++) t.emplace_back([&] { int w; q.get(3, &w, [&](int* out) { made++; *out = 1; return true; }); });
  for (auto& x : t) x.join();
  return made == 1 ? 0 : 9;
}
"""


def test_once_for_each_device(tmp_path):
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "mxfp8_quantization_amax_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", inc, "-o", str(exe), str(src)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


UPDATES = r"""
#include "per_device.h"

int main() {
  fp8q::PerDevice<int> p;
  int seen = -1;
  auto add = [&](int n) { return [&seen, n](int* v) { seen = *v; *v += n; }; };
  p.update(2, add(5));
  if (seen != 0) return 1;
  p.update(2, add(1));
  if (seen != 5) return 2;
  p.update(3, add(1));
  if (seen != 0) return 3;
  p.update(2, add(0));
  if (seen != 6) return 4;
  p.update(64, add(9));
  p.update(64, add(9));
  return seen == 0 ? 0 : 5;
}
"""


def test_updates_are_each_device_s_own(tmp_path):
    src, exe = tmp_path / "t.cc", tmp_path / "t"
    src.write_text(UPDATES)
    inc = os.path.join(ROOT, "mxfp8_quantization_amax_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", inc, "-o", str(exe), str(src)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
