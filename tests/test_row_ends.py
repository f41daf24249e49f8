"""The rule that says which groups over a row's ends are copied whole: no such copy leaves the tensor, whatever its
rows' number, width, stride and alignment (compiled here with g++; no GPU)."""
import os
import subprocess

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "routing_shared_expert_gb300", "csrc")

# Every group that a row fills in part, as the kernels enumerate them: the rows' first elements lie
# (phase + row * ld) % G elements into a group.
PROGRAM = r"""
#include "row_ends.h"
#include <cstdio>
int main() {
  long whole = 0, single = 0;
  for (int G = 4; G <= 8; G += 4)
    for (int T = 1; T <= 20; ++T)
      for (int d = 1; d <= 2 * G + 1; ++d)
        for (int ld = d; ld <= d + G + 1; ++ld)
          for (int phase = 0; phase < G; ++phase)
            for (int row = 0; row < T; ++row) {
              const long first = static_cast<long>(row) * ld, end = static_cast<long>(T - 1) * ld + d;
              const int room = moe::rows_of_room(ld, G), shift = static_cast<int>((phase + first) % G);
              for (int c = -shift; c < d; c += G) {
                unsigned mask = 0;
                for (int j = 0; j < G; ++j)
                  if (c + j >= 0 && c + j < d) mask |= 1u << j;
                if (mask == (1u << G) - 1 || mask == 0) continue;
                if (!moe::copied_whole(row, T, room, mask, G)) {
                  ++single;
                  // rows that are not short: only the tensor's own ends
                  if (ld >= G - 1 && first + c >= 0 && first + c + G <= end && row > 0 && row < T - 1) return 2;
                  continue;
                }
                ++whole;
                if (first + c < 0 || first + c + G > end) {
                  std::printf("G %d T %d d %d ld %d phase %d row %d column %d\n", G, T, d, ld, phase, row, c);
                  return 1;
                }
              }
            }
  return whole > 0 && single > 0 ? 0 : 3;
}
"""


def test_no_copied_group_leaves_the_tensor(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_the_kernels_copy_by_the_rule():
    """Every copy of a partly filled group asks the rule, with the room of all operands that are read."""
    with open(os.path.join(CSRC, "layernorm.cuh")) as fh:
        body = fh.read()
    assert "s.part[k] && copied_whole(at, T, room, s.mask[k], G)" in body and body.count("copy_whole<G>") == 1
    for name, copies in (("layernorm.cu", 2), ("layernorm_grad.cuh", 3)):
        with open(os.path.join(CSRC, name)) as fh:
            text = fh.read()
        assert text.count("ahead, T, a.room)") == copies == text.count(".copy(") and "a.room = room_of(" in text
