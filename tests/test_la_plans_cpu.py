"""The time-cut plans that the parity tests of test_la_plans_gpu are there for, from the planner itself: whole
units beside cut ones, in the forward and over both directions of the backward."""

import os
import subprocess

import pytest

from mamba_selective_scan_fwd_gb300 import build

SHAPES = [  # Bsz, L, H, G, N, P
    (2, 2500, 160, 16, 16, 8),
    (2, 2500, 160, 20, 72, 8),
    (1, 2300, 310, 31, 128, 16),
]

SOURCE = """
#include <cstdio>
#include "lm/la_tc.h"
using namespace ss::la;
int main(int argc, char** argv) {
    long v[4];
    while (scanf("%ld %ld %ld %ld", v, v + 1, v + 2, v + 3) == 4) {
        const long units = v[0] * v[2] * ((v[3] + kTileP - 1) / kTileP);
        for (int dirs = 1; dirs <= 2; dirs++) {
            const TcPlan p = tc_plan(dirs * units, v[1], dirs == 1 ? 2 * kSms : kSms);
            printf("%ld %ld %ld %ld\\n", (long)p.whole, (long)p.cut, (long)p.K, (long)p.seg);
        }
    }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cu").write_text(SOURCE)
    exe = str(d / "plan")
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I", build.CSRC, "-o", exe, str(d / "plan.cu")], check=True)
    text = "".join(f"{b} {L} {H} {P}\n" for b, L, H, _, _, P in SHAPES)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
    rows = [tuple(map(int, out[i:i + 4])) for i in range(0, len(out), 4)]
    return {s: {"fwd": rows[2 * i], "bwd": rows[2 * i + 1]} for i, s in enumerate(SHAPES)}


@pytest.mark.parametrize("way", ["fwd", "bwd"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_whole_units_beside_cut_ones(plans, shape, way):
    whole, cut, K, seg = plans[shape][way]
    assert whole > 0 and cut > 0 and K > 2
    assert (K - 1) * seg < shape[1] <= K * seg
    units = shape[0] * shape[2] * -(-shape[5] // 64)
    assert whole + cut == units * (2 if way == "bwd" else 1)
    if way == "bwd":  # the reverse direction's last units are the cut ones, its first are whole
        assert whole > units
