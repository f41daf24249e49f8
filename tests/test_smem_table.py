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


LIMITS = r"""
#include "smem_table.h"
#include <initializer_list>
enum Error { kOk, kFailed };
int main() {
  // kernels of the library on eight devices: all have entries
  static moe::SmemTable t;
  for (int d = 0; d < 8; ++d)
    for (int f = 0; f < KERNELS; ++f)
      if (!t.find(reinterpret_cast<char*>(1 << 20) + 16 * f, d)) return 1;
  // one kernel and its limit as the driver keeps it; with an entry and, the table full, without
  moe::SmemTable::Entry own{nullptr, 0, 0};
  for (auto* e : {&own, static_cast<moe::SmemTable::Entry*>(nullptr)}) {
    size_t limit = 0;
    int sets = 0;
    auto get = [&](size_t* held) { return *held = limit, kOk; };
    auto set = [&](size_t bytes) { return limit = bytes, ++sets, kOk; };
    const size_t asked[] = {50000, 200000, 60000, 200000, 48000, 220000, 50000};
    size_t most = 0;
    for (size_t bytes : asked) {
      if (moe::raise_limit<Error>(e, bytes, get, set) != kOk || limit < bytes || limit < most) return 2;
      most = limit;
    }
    if (sets != 3) return 3;
    // a refused limit stays an error at the next call too
    auto refuse = [&](size_t) { return kFailed; };
    for (int i = 0; i < 2; ++i)
      if (moe::raise_limit<Error>(e, 230000, get, refuse) != kFailed || limit != 220000) return 4;
  }
  auto broken = [&](size_t*) { return kFailed; };
  auto set = [&](size_t) { return kOk; };
  return moe::raise_limit<Error>(nullptr, 1, broken, set) == kFailed ? 0 : 5;
}
"""


def test_limits_never_fall(tmp_path):
    """With 400 kernels on eight devices every one has an entry, and past a full table a smaller plan does not take
    back what a larger one set."""
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(LIMITS.replace("KERNELS", "400"))
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
    with open(os.path.join(CSRC, "gemm_tc.cu")) as fh:
        body = re.search(r"cudaError_t set_smem_once\(.*?\n}\n", fh.read(), re.S).group(0)
    assert body.index("lock_guard") < body.index("raise_limit")


def test_the_kernels_own_arrays_count():
    """The normalisation raises a kernel's limit wherever the plan's bytes and the kernel's own arrays can pass the 48 KB
    that every kernel has; the arrays' size is held to what the launch counts on."""
    def text(name):
        with open(os.path.join(CSRC, name)) as fh:
            return re.sub(r"//[^\n]*", "", fh.read())

    plan = text("layernorm.cuh")
    static = eval(re.search(r"kStaticSmem = ([\d* ]+);", plan).group(1))
    default = eval(re.search(r"kDefaultSmem = ([\d* ]+);", plan).group(1))
    assert (static, default) == (4096, 49152) and "bytes + kStaticSmem > kDefaultSmem ? set_smem_once" in plan
    teams = int(re.search(r"kMaxTeams = (\d+)", plan).group(1))
    for name, most in (("layernorm.cu", teams * 2 * 32 * 2 * 4), ("layernorm_grad.cuh", teams * 2 * 32 * 4)):
        body = text(name)
        assert most <= static and "static_assert(sizeof(part) <= kStaticSmem" in body
