"""The tree attention's load order on the host (csrc/tree_ring.cuh, compiled with the host compiler): which ring
positions a segment's tiles have, and which copies the load warp waits for at its end, also when one of its waits has
run out anywhere on the way. No GPU."""
import os
import subprocess

import pytest

from shared_kv_draft_b200.build import SRC_DIR

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "tree_ring.cuh"
using namespace orthrus;

static void want(bool ok, const char* what) {
  if (!ok) { printf("%s\n", what); exit(1); }
}

int main() {
  // every tile of a segment has one position of K and one of V; K runs `ahead` tiles ahead of V
  for (int ahead = 2; ahead <= 4; ahead += 2)
    for (int nt = 1; nt < 40; ++nt) {
      std::vector<int> used(2 * nt, 0);
      for (int k = 0; k < nt; ++k) {
        want(tree_pos_k(k, ahead) < 2u * nt && tree_pos_v(k, ahead, nt) < 2u * nt, "position outside the segment");
        ++used[tree_pos_k(k, ahead)];
        ++used[tree_pos_v(k, ahead, nt)];
        if (k + ahead < nt) want(tree_pos_k(k + ahead, ahead) == tree_pos_v(k, ahead, nt) + 1, "K does not follow V");
      }
      for (int u : used) want(u == 1, "a position is not used exactly once");
    }
  // a CTA with `segs` segments of nt tiles whose load warp gives up at one of its waits (`fail` counts them, q's
  // among them; or never): it waits for phases that its copies complete, each stage's last one among them, and
  // for no others
  for (unsigned stages = 10; stages <= 20; stages += 10)
    for (int segs = 0; segs < 4; ++segs)
      for (int nt = 1; nt < 14; nt += 3)
        for (int fail = 0; fail <= segs * (2 * nt + 1); ++fail) {
          const int lead = nt < 4 ? nt : 4;
          std::vector<unsigned> phases(stages, 0);  // of full[s], that copies complete
          unsigned qs = 0, seg = 0, base = 0;       // q's copies; the warp's counts
          int waits = 0;
          bool ok = true;
          for (int s = 0; s < segs; ++s) {
            if (ok)
              for (int p = 0; p < 2 * nt; ++p) {
                if (p == lead) {
                  if (!(ok = waits++ != fail)) { base += p; break; }
                  ++qs;
                }
                if (!(ok = waits++ != fail)) { base += p; seg += p >= lead ? 1 : 0; break; }
                ++phases[(base + p) % stages];
              }
            if (ok) { base += 2 * nt; ++seg; }
          }
          want(seg == qs, "count of q copies");
          std::vector<char> seen(stages, 0);
          for (unsigned k = tree_pos_last(base, stages); k < base; ++k) {
            want(k / stages + 1 == phases[k % stages], "waits for a phase that is not the stage's last copy's");
            seen[k % stages] = 1;
          }
          for (unsigned s = 0; s < stages; ++s) want(seen[s] == (phases[s] > 0), "a copy is not waited for");
        }
  puts("ok");
}
"""


@pytest.mark.parametrize("flags", [["-O2"], ["-O1", "-fsanitize=undefined", "-fno-sanitize-recover"]], ids=["plain", "ubsan"])
def test_ring_positions_and_closing_waits(tmp_path, flags):
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", *flags, "-I", SRC_DIR, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


def test_the_load_warp_counts_what_it_issued():
    """The kernel's load warp keeps the counts as above: they stand still after a wait that has run out, and the
    closing loop ends at the first wait that does."""
    with open(os.path.join(SRC_DIR, "tree_attention.cuh")) as f:
        text = " ".join(f.read().split())
    for part in ("base += p; break; }", "base += p; seg += p >= lead ? 1 : 0; break; }", "if (ok) { base += 2 * nt; ++seg; }",
                 "k = tree_pos_last(base, S::kStages); landed && k < base; ++k"):
        assert part in text, part
