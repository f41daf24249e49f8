"""Groups of values: a size that a type does not come in does not compile, so that none can drop its values in silence
(compiled here with nvcc; no GPU)."""
import importlib.util
import os
import subprocess

import pytest

from tests.conftest import ROOT

spec = importlib.util.spec_from_file_location("_moe_build", os.path.join(ROOT, "routing_shared_expert_gb300", "build.py"))
build = importlib.util.module_from_spec(spec)
spec.loader.exec_module(build)

PROGRAM = """
#include "vec8.cuh"
__global__ void k(VALUE* p) {
  float2 v[PAIRS];
  moe::read_group(reinterpret_cast<const char*>(p), p, v);
  moe::store_whole(p, v);
}
"""


@pytest.mark.parametrize("t,n,fits", [("__nv_bfloat16", 4, True), ("__nv_bfloat16", 2, True), ("float", 2, True),
                                      ("float", 4, False)])
def test_groups(tmp_path, t, n, fits):
    src = tmp_path / "t.cu"
    src.write_text(PROGRAM)
    r = subprocess.run([build.nvcc(), *build.ARCH, *build.CFLAGS, f"-DVALUE={t}", f"-DPAIRS={n}", "-c", str(src), "-o",
                        str(tmp_path / "t.o")], capture_output=True, text=True)
    assert (r.returncode == 0) == fits and fits == ("no instance of overloaded function" not in r.stderr), r.stderr
