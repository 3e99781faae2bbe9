"""The ring of r.P distances of the band kernel of relattn_extend, on the CPU: the
kernel's own arithmetic (csrc/extend_ring.h), compiled for the host and run over
every place that an item's first step can have.  At an item's start the two threads
of a row store their halves of up to three chunks without waiting for each other, so
halves of different threads must not share a slot, and every distance that the first
step reads (none is read below 0) must lie in its slot afterwards."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "relative_position_biased_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "extend_ring.h"
using namespace relattn;

int main() {
  int bad = 0;
  long cases = 0;
  for (int wide = 0; wide < 2; ++wide) {
    const int slots = wide ? 6 : 5, most = wide ? 64 : 32;
    for (int tokens = 1; tokens <= most; ++tokens)
      for (int D0 = 1 - tokens; D0 < 64 * 7; ++D0)       // (the last row sees the step's first key)
        for (int before = 0; before < 3; ++before, ++cases) {      // chunks that the CTA took before
          const BandChunks c = band_chunks(D0, tokens);
          int owner[6] = {-1, -1, -1, -1, -1, -1}, held[6] = {-1, -1, -1, -1, -1, -1};
          bool shared = false;
          for (int x = c.start; x <= c.first; ++x)
            for (int half = 0; half < 2; ++half) {
              if (!@STORED@) continue;
              const int s = band_slot(before + x - c.start, half, slots);
              shared |= owner[s] >= 0 && owner[s] != half;
              owner[s] = half;
              held[s] = 2 * x + half;
            }
          bool lost = false;
          for (int d = D0 - 63 > 0 ? D0 - 63 : 0; d < D0 + tokens; ++d)
            lost |= held[band_slot(before + (d >> 6) - c.start, (d >> 5) & 1, slots)] != d >> 5;
          bad += shared || lost;
        }
  }
  std::printf("%ld %d\n", cases, bad);
}
"""


def run(tmp_path, stored):
    cxx = shutil.which("g++") or pytest.skip("no host compiler")
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM.replace("@STORED@", stored))
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    cases, bad = (int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert cases > 100000
    return bad


def test_halves_stored_at_an_items_start_share_no_slot_and_are_all_that_is_read(tmp_path):
    assert run(tmp_path, "band_stored(x, half, c.first, slots)") == 0


def test_storing_every_half_would_let_an_older_one_come_last(tmp_path):
    assert run(tmp_path, "true") > 0
