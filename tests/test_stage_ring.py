"""The bookkeeping of a ring of copies (csrc/stage_ring.h) against a model of its barriers, on the host: what a kernel
waits for on its way out when a wait has run out, as nothing may make that happen on a GPU."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "conv_bn_activation_gb300", "csrc")

# A barrier of a stage: copies in flight complete its current phase; a wait with a parity succeeds once the phase of that
# parity is complete.  Pieces of any number of steps, the copies of step + STAGES - 1 issued before the wait for `step`.
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "stage_ring.h"

struct Barrier {
  unsigned done = 0;  // phases completed
  bool in_flight = false;
  bool complete(unsigned parity) const { return ((done & 1u) ^ 1u) == parity; }  // the last completed one has that parity
  void land() { in_flight = false, ++done; }
};

template <int STAGES>
int walk(unsigned seed, int fail_at) {  // the fail_at-th wait runs out: 0 as it has to be
  srand(seed);
  Barrier bar[STAGES];
  cb::StageRing<STAGES> ring;
  int waits = 0;
  for (int piece = 0; piece < 6; ++piece) {
    const int steps = rand() % 7;
    int stage = 0;
    auto issue = [&](int step, int at) {
      if (step >= steps) return 0;
      if (bar[at].in_flight) return 1;  // a stage that still takes copies
      bar[at].in_flight = true;
      return 0;
    };
    for (int s = 0; s + 1 < STAGES; ++s)
      if (issue(s, s)) return 1;
    for (int step = 0; step < steps; ++step) {
      if (issue(step + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1)) return 2;
      if (bar[stage].complete(ring.parity(stage))) return 3;  // would not wait for the copies
      if (waits++ == fail_at) {
        std::vector<int> asked(STAGES, 0);
        bool bad = false;
        ring.in_flight(stage, step, steps, [&](int s, unsigned parity) {
          ++asked[s];
          bad |= bar[s].complete(parity);  // returns at once, with the copies in flight
          if (bar[s].in_flight) bar[s].land();
          bad |= !bar[s].complete(parity);  // waits for what does not come
        });
        for (int s = 0; s < STAGES; ++s) bad |= asked[s] > 1 || bar[s].in_flight;
        return bad ? 4 : 0;
      }
      bar[stage].land();
      if (!bar[stage].complete(ring.parity(stage))) return 5;
      ring.waited(stage);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
  }
  return 0;
}

int main() {
  for (unsigned seed = 0; seed < 200; ++seed)
    for (int fail = -1; fail < 30; ++fail) {
      const int r[3] = {walk<2>(seed, fail), walk<3>(seed, fail), walk<4>(seed, fail)};
      for (int i = 0; i < 3; ++i)
        if (r[i]) return printf("%d stages, seed %u, wait %d: %d\n", i + 2, seed, fail, r[i]), 1;
    }
  return 0;
}
"""


def test_what_is_in_flight_when_a_wait_runs_out(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    (tmp_path / "walk.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, str(tmp_path / "walk.cpp"), "-o", str(tmp_path / "walk")], check=True)
    r = subprocess.run([str(tmp_path / "walk")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_the_decode_over_4_bits_drains_by_it():
    """A failed wait turns no phase, and what is drained is what the ring names."""
    with open(os.path.join(CSRC, "decode4.cuh")) as f:
        code = f.read()
    assert "if (alive) flight.waited(stage);" in code and code.count("mbar_wait_drain(") == 1
    assert "flight.in_flight(stage, step, steps" in code
