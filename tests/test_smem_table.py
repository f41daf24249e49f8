"""The host table of shared-memory limits: every kernel of the library on several devices has its own
entry, so that none asks the driver again at each call (compiled here with g++; no GPU)."""
import os
import re
import subprocess

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "routing_shared_expert_gb300", "csrc")

PROGRAM = r"""
#include "smem_table.h"
#include <cstdio>
int main() {
  static moe::SmemTable t;
  static char kernels[4096];
  const int funcs = KERNELS, devs = 4;
  for (int round = 0; round < 3; ++round)
    for (int d = 0; d < devs; ++d)
      for (int f = 0; f < funcs; ++f) {
        auto* e = t.find(kernels + 16 * f, d);
        if (!e || e->func != kernels + 16 * f || e->dev != d) return 1;
        if (e->bytes != (round ? static_cast<size_t>(1000 * d + f + round - 1) : 0)) return 2;
        e->bytes = static_cast<size_t>(1000 * d + f + round);
      }
  // past its slots it gives none, and keeps what it has
  int full = 0;
  for (int f = 0; f < 4096; ++f) full += t.find(reinterpret_cast<char*>(1 << 20) + f, 9) == nullptr;
  if (full != 4096 - (static_cast<int>(moe::SmemTable::kSlots) - funcs * devs)) return 3;
  return t.find(kernels, 0)->bytes == 2 ? 0 : 4;
}
"""


def test_every_kernel_has_an_entry(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM.replace("KERNELS", "200"))
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_the_limit_setter_uses_it():
    with open(os.path.join(CSRC, "gemm_tc.cu")) as fh:
        body = re.search(r"cudaError_t set_smem_once\(.*?\n}\n", fh.read(), re.S).group(0)
    assert "SmemTable" in body and "[64]" not in body
