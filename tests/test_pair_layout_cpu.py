"""The shared-memory map of the MLA over CTA pairs, checked on the host: areas that are in use at the same time by
warps no barrier keeps apart must not overlap."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_attention_06_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "mla_pair_layout.h"
using namespace dsa::packed;
int main() {
  for (int v = 0; v < 2; ++v)
    for (int w = 0; w < kSoftmaxWarps; ++w) {
      std::printf("p %d %d %d %d\n", v, w, p_offset(v, w), kWarpPBytes);
      std::printf("stage %d %d %d %d\n", v, w, stage_offset(v, w), kStageBytes);
    }
  const int map[][2] = {{OFF_Q, kSmemQ * Q_CHUNK}, {OFF_P, 2 * P_BYTES}, {OFF_Y, kYBlocks * K_CHUNK}, {OFF_X, kXBlocks * K_CHUNK},
                        {OFF_V, 3 * V_BYTES}, {OFF_BAR, NBAR * 8}, {OFF_MASK, kSlots * 8}, {OFF_POISON, kSlots * 8},
                        {OFF_STATS, kRows * 4}, {OFF_MAX, 2 * kRows * 4}, {OFF_UNIT, kUnitSlots * kUnitBytes},
                        {OFF_ROWS, kSlots * 2 * kTile * 4}, {OFF_MAIL, 16}, {OFF_MISC, 16}, {SMEM, 0}};
  for (const auto& a : map) std::printf("map 0 0 %d %d\n", a[0], a[1]);
  std::printf("fill 0 0 %d %d\n", OFF_V, kFillWarps * kStageBytes);
  std::printf("own 0 0 %d %d\n", OFF_V, 2 * V_BYTES);
  std::printf("area 0 0 %d %d\n", OFF_P, P_BYTES);
  std::printf("area 1 0 %d %d\n", OFF_P + P_BYTES, P_BYTES);
}
"""


@pytest.fixture(scope="module")
def areas(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("layout")
    src, exe = d / "layout.cpp", d / "layout"
    src.write_text(PROGRAM)
    subprocess.check_call([cxx, "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)])
    out = {}
    for line in subprocess.check_output([str(exe)], text=True).splitlines():
        name, *n = line.split()
        v, w, at, size = map(int, n)
        out.setdefault(name, []).append((v, w, at, at + size))
    return out


def overlap(a, b):
    return a[2] < b[3] and b[2] < a[3]


def test_a_warp_stages_its_outputs_in_no_other_warps_rows(areas):
    # one softmax warp may write P of the next unit while another still stages outputs of the last
    for s in areas["stage"]:
        for other in areas["p"] + areas["stage"]:
            if (s[0], s[1]) != (other[0], other[1]):
                assert not overlap(s, other), (s, other)


def test_p_rows_lie_side_by_side_in_their_ctas_area(areas):
    for v in range(2):
        mine = [p for p in areas["p"] if p[0] == v]
        assert [p[1] for p in mine] == list(range(len(mine)))
        at = areas["area"][v][2]
        for p in mine:
            assert p[2] == at
            at = p[3]
        assert at == areas["area"][v][3]


def test_areas_follow_each_other(areas):
    m = areas["map"]
    for a, b in zip(m, m[1:]):
        assert a[3] <= b[2]
    # the fill warps, which help with a CTA's last unit, stage where the own page's values were
    assert areas["fill"][0][3] <= areas["own"][0][3]
