"""Whether two tensors of a list share memory: exact, against the bytes themselves (compiled here with g++), and as the
clipping call applies it (no GPU)."""
import ctypes
import os
import subprocess

import pytest

from tests.conftest import ROOT, ensure_built

CSRC = os.path.join(ROOT, "routing_shared_expert_gb300", "csrc")

PROGRAM = r"""
#include "share_memory.h"
#include <cstdio>
#include <random>
using moe::Reach;
static Reach at(uint64_t lo, uint64_t rows, uint64_t width, uint64_t pitch, bool written = true) {
  return moe::reach_of(reinterpret_cast<void*>(lo), rows, width, pitch, written);
}
int main() {
  std::mt19937 rng(1);
  auto pick = [&](int lo, int hi) { return lo + static_cast<int>(rng() % (hi - lo + 1)); };
  long shared = 0, apart = 0, woven = 0;
  for (int i = 0; i < 400000; ++i) {
    Reach r[2];
    bool byte[2][2048] = {};
    for (int k = 0; k < 2; ++k) {
      const int rows = pick(1, 12), width = pick(1, i % 3 ? 6 : 40), pitch = width + pick(0, i % 2 ? 60 : 8), lo = pick(1, 300);
      r[k] = at(lo, rows, width, pitch);
      for (int j = 0; j < rows; ++j)
        for (int c = 0; c < width; ++c) byte[k][lo + j * pitch + c] = true;
    }
    bool want = false;
    for (int c = 0; c < 2048; ++c) want = want || (byte[0][c] && byte[1][c]);
    if (moe::share_memory(r[0], r[1]) != want || moe::share_memory(r[1], r[0]) != want) {
      for (const Reach& e : r) std::printf("%lu %lu %lu %lu\n", (long)e.lo, (long)e.hi, (long)e.pitch, (long)e.width);
      return 1;
    }
    (want ? shared : apart) += 1;
    woven += !want && r[0].lo < r[1].hi && r[1].lo < r[0].hi;
    // a third tensor in the list, read only: what counts is whether a written one is met
    std::vector<Reach> list = {r[0], at(1500, 1, 8, 8, false), r[1], at(1500, 1, 8, 8, false)};
    if (moe::any_written_is_shared(list) != want) return 2;
  }
  if (shared < 1000 || apart < 1000 || woven < 1000) return 3;
  // the largest sizes: rows 2^40 elements apart in all, strides that differ by one element
  const uint64_t base = uint64_t{1} << 20, n = uint64_t{1} << 20, p = uint64_t{1} << 20;
  // 4 bytes of pitch apart: row k of the second begins 4 k bytes further into the first's gaps
  if (moe::share_memory(at(base, n, 4, p), at(base + 4, 1 << 17, 4, p + 4))) return 4;
  if (!moe::share_memory(at(base, n, 4, p), at(base + 4, n, 4, p + 4))) return 5;      // once round
  if (!moe::share_memory(at(base, n, 4, p), at(base + 8, n, 4, 2 * p - 4))) return 6;
  if (moe::share_memory(at(base, n, 4, p), at(base + 8, n / 2, 4, 2 * p))) return 7;
  if (moe::floor_sum(uint64_t{1} << 40, 1, 0, 5) != 5 * (uint64_t{1} << 40)) return 8;
  return 0;
}
"""


def test_against_the_bytes(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout)


@pytest.fixture(scope="module")
def clip():
    """The status of a clipping call whose workspace is too small: -4 for a list that is allowed, so that nothing is
    enqueued."""
    ensure_built()
    from routing_shared_expert_gb300 import _native as nat

    def call(grads, out=None, norm=0x10000, size=256):
        lists = [(nat.moe_tensor * len(x))(*[nat.moe_tensor(*t) for t in x]) if x else None for x in (grads, out)]
        return nat.library().moe_clip_grad_norm(*lists, len(grads), 1.0, ctypes.c_void_p(norm),
                                                ctypes.c_void_p(0x20000), size, None)
    return call


A = 0x100000


@pytest.mark.parametrize("pair", [
    ((A, 4, 8, 16, 0), (A + 32, 1, 8, 0, 0)),            # one row in the gap of a matrix
    ((A, 4, 8, 16, 0), (A + 96, 1, 8, 0, 0)),
    ((A, 4, 8, 16, 0), (A + 32, 2, 8, 32, 0)),           # every second gap
    ((A, 4, 8, 16, 0), (A + 32, 3, 2, 18, 0)),           # another stride, moving through the gaps
    ((A, 4, 8, 16, 0), (A + 32, 4, 2, 19, 0)),           # values 8, 27, 46 in gaps and 65 behind the last row, 48 to 55
    ((A, 4, 8, 16, 0), (A + 32, 1, 16, 0, 1)),           # bf16 in the gap
    ((A, 2, 4, 100, 0), (A + 40, 5, 8, 8, 0)),           # a dense matrix in the gap
])
def test_lists_that_share_nothing_are_allowed(clip, pair):
    assert clip(list(pair)) == -4 and clip(list(pair[::-1])) == -4


@pytest.mark.parametrize("pair", [
    ((A, 4, 8, 16, 0), (A + 32, 1, 9, 0, 0)),            # one value into the next row
    ((A, 4, 8, 16, 0), (A + 28, 1, 8, 0, 0)),
    ((A, 4, 8, 16, 0), (A + 32, 2, 8, 17, 0)),
    ((A, 4, 8, 16, 0), (A + 32, 3, 2, 21, 0)),           # values 8, 29 and 50, the last in the row from 48
    ((A, 4, 8, 16, 0), (A + 32, 1, 18, 0, 1)),
])
def test_lists_that_share_memory_are_refused(clip, pair):
    assert clip(list(pair)) == -1 and clip(list(pair[::-1])) == -1


def test_refused_whatever_the_workspace(clip):
    """The check of the list comes before that of the workspace, so that the cases above reach it."""
    assert clip([(A, 1, 8, 0, 0), (A, 1, 8, 0, 0)]) == -1


def test_the_norm_lies_in_no_tensor(clip):
    """It is written before the gradients are read for the second time."""
    grads, out = [(A, 4, 8, 16, 0)], [(A + 0x1000, 4, 8, 16, 0)]
    for norm in (A, A + 28, A - 4, A + 3 * 64 + 24, A + 0x1000, A + 0x1000 + 64):
        assert clip(grads, out, norm, 1 << 40) == -1
    assert clip(grads, None, A + 8, 1 << 40) == -1
