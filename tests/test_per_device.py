"""Counts that the host asks of each device once (csrc/per_device.h), in a small host program."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "latent_moe_decode_gb300", "csrc")

PROGRAM = r"""
#include "per_device.h"
#include <cstdio>
int asked = 0;
moe::PerDevice<9> counts;
int get(int device, int i, int answer) { return counts.get(device, i, [&] { ++asked; return answer; }); }
#define HOLDS(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
  HOLDS(get(0, 8, -1) == -1 && asked == 1);             // a query that fails is asked again
  HOLDS(get(0, 8, 17) == 17 && asked == 2);
  HOLDS(get(0, 8, 99) == 17 && asked == 2);             // known
  HOLDS(get(1, 8, 15) == 15 && asked == 3);             // each device has its own
  HOLDS(get(0, 4, 0) == 0 && get(0, 4, 5) == 0 && asked == 4);  // nothing is an answer, too
  HOLDS(get(0, 8, 1) == 17 && get(1, 8, 1) == 15 && asked == 4);
  HOLDS(get(63, 0, 2) == 2 && get(64, 0, 2) == -1 && get(-1, 0, 2) == -1 && get(0, 9, 2) == -1);
  return 0;
}
"""


def test_per_device(tmp_path):
    (tmp_path / "main.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(tmp_path / "main.cpp"), "-o", str(tmp_path / "main")], check=True)
    run = subprocess.run([str(tmp_path / "main")], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout


def test_the_products_ask_each_device():
    """No count of resident clusters of the products is kept for the process."""
    for name in ("linear_narrow.cu", "fp8_gemm_narrow.cu"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert "static PerDevice<kMaxSplits + 1>" in text and "static std::atomic<int>" not in text, name
