"""By which kernel a forward product runs (CPU only): the rules of product.hpp, compiled for the host alone, asked for the
sizes at which the GPU tests check each of them."""
import os
import subprocess

import pytest

from equivariant_edge_convolution_amd import binding as B
from equivariant_edge_convolution_amd.build import CSRC, HIPCC
from test_gpu_gated_paths import PATHS

PROGRAM = r"""
#include <cstdio>
#include "product.hpp"
using namespace eec;
int main() {
  const char* names[] = {"SMALL", "GENERAL", "TILE64", "TILE128", "TILE128X2", "TILE256", "PARTED", "FEW"};
  static_assert(FEW == 7 && SMALL == 0 && TILE64 == 2 && TILE256 == 5, "names in order");
  long rows, inner, outer;
  int dtype, out, gated;
  while (scanf("%ld %ld %ld %d %d %d", &rows, &inner, &outer, &dtype, &out, &gated) == 6) {
    const FwdPlan f = fwd_plan(rows, outer, inner, dtype, out, gated);
    const bool aligned = dtype != EEC_F32 && inner * packed_size(dtype) % 16 == 0;
    const Plan p = plan_product(rows, gated ? gated_columns(outer) : outer, inner, dtype, aligned || f.packed, f.packed, true);
    printf("%s %d %d\n", names[p.kind], f.packed, p.splits > 1);
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plans")
    (d / "plans.hip").write_text(PROGRAM)
    r = subprocess.run([HIPCC, "--offload-host-only", "-x", "hip", "-std=c++17", "-O1", "-I", CSRC, str(d / "plans.hip"), "-o",
                        str(d / "plans")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    lines = [f"{rows} {inner} {outer} {B.DTYPES[dt]} {B.DTYPES[dt] if B.DTYPES[dt] < 3 else 2} {int(gated)}" for dt, gated, rows, inner, outer, *_ in PATHS]
    out = subprocess.run([str(d / "plans")], input="\n".join(lines), capture_output=True, text=True, check=True).stdout.split("\n")
    return dict(zip(((p[0], *p[1:5]) for p in PATHS), out))


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(str(v).replace("torch.", "") for v in p))
def test_the_size_takes_the_path(plans, path):
    dt, gated, rows, inner, outer, kernel, packed, split = path
    assert plans[(dt, gated, rows, inner, outer)] == f"{kernel} {int(packed)} {int(split)}"


def test_every_kernel_has_a_size():
    for kinds, gated in ((("TILE64", "TILE128", "TILE128X2", "TILE256"), True), (("SMALL", "GENERAL"), True)):
        for k in kinds:
            types = {p[0] for p in PATHS if p[5] == k and p[1] == gated}
            assert len(types) >= (4 if k.startswith("TILE") else 2), k
