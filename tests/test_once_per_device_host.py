"""What kernels set up once on each device (csrc/gla_once.cuh), on the CPU: every device gets it, a failure is
not taken for done."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_recurrence_simple_gb300", "csrc")

SOURCE = r"""
#include <initializer_list>
#include "gla_once.cuh"
static int current, failing;
struct Fake {
  using Error = int;
  static constexpr int kSuccess = 0;
  static int device(int& d) { d = current; return failing; }
};
int main() {
  static gla::OncePerDevice<Fake> once;
  int runs[70] = {}, result = 9;
  auto go = [&](int dev) { current = dev; return once([&] { ++runs[dev]; return result; }); };
  if (go(0) != 9 || go(0) != 9 || runs[0] != 2) return 1;   // failures are tried again
  result = 0;
  for (int i = 0; i < 3; ++i)
    for (int dev : {0, 1, 63, 64}) if (go(dev) != 0) return 2;
  if (runs[0] != 3 || runs[1] != 1 || runs[63] != 1 || runs[64] != 3) return 3;
  failing = 5;
  if (go(1) != 5 || runs[1] != 1) return 4;
  return 0;
}
"""


def test_every_device_is_set_up_once(tmp_path):
    (tmp_path / "once.cpp").write_text(SOURCE)
    exe = str(tmp_path / "once")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-o", exe, str(tmp_path / "once.cpp")], check=True)
    assert subprocess.run([exe], timeout=60).returncode == 0


def test_no_source_keeps_one_flag_for_all_devices():
    """A static truth value beside cudaFuncSetAttribute would let the second device's first launch fail."""
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        assert "static bool" not in text, name
