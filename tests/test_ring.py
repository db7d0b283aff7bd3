"""The copies in flight of a ring of slots land before its CTA exits (csrc/ring.cuh): the waits that drain_ring makes,
against a model of the barriers on the CPU (compiled with nvcc, no GPU call)."""
import os
import shutil
import subprocess

import pytest

from joint_attention_gb300.build import CSRC

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "ring.cuh"

// A barrier whose phases complete in turn.  A wait for a parity returns at once if the last completed phase has it
// (before any has completed: parity 1), else it stays until that phase completes, or runs out its limit.
struct Barrier {
  int phases = 0;  // completed
  bool blocks(uint32_t parity) const { return static_cast<uint32_t>(phases & 1) == parity; }
};

int main() {
  int fails = 0;
  auto expect = [&](bool ok, const char* what, int slots, int issued) {
    if (!ok && ++fails < 9) std::printf("%s: %d slots, %d issued\n", what, slots, issued);
  };
  std::srand(1);
  for (int slots = 1; slots <= 8; ++slots)
    for (int issued = 0; issued <= 5 * slots; ++issued) {
      // Copies that complete on another CTA's barriers: one wait or more, none of which returns at once.
      {
        std::vector<Barrier> own(slots);
        int waits = 0, at_once = 0;
        jattn::drain_ring(issued, slots, false, [&](int s, uint32_t parity) {
          ++waits;
          if (!own[s].blocks(parity)) ++at_once;
        });
        expect(at_once == 0, "a wait of the second CTA returns at once", slots, issued);
        expect((waits > 0) == (issued > 0), "the second CTA waits if it has copies", slots, issued);
      }
      // On this CTA's: for every choice of the last copies that have not landed, each is waited for.
      for (int trial = 0; trial < 32; ++trial) {
        std::vector<Barrier> own(slots);
        std::vector<char> late(issued, 0), met(issued, 0);
        for (int i = 0; i < issued; ++i) {
          late[i] = i >= issued - slots && std::rand() % 2;  // a slot is filled again only once its copy has landed
          if (!late[i]) ++own[i % slots].phases;
        }
        jattn::drain_ring(issued, slots, true, [&](int s, uint32_t parity) {
          if (!own[s].blocks(parity)) return;
          for (int i = 0; i < issued; ++i)
            if (late[i] && i % slots == s) met[i] = 1;
        });
        for (int i = 0; i < issued; ++i) expect(late[i] == met[i], "a copy in flight is waited for", slots, issued);
      }
    }
  std::printf(fails ? "FAILED\n" : "ring ok\n");
  return fails != 0;
}
"""


def test_drain_ring_waits_for_every_copy_in_flight(tmp_path):
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "ring.cu", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and "ring ok" in r.stdout, r.stdout
