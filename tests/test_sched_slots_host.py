"""The prefill's counter slots on the host: a launch that fails behind a kernel
that is queued already still uses its slot up. csrc/sched_slots.cuh is compiled
as plain C++ against a fake of the CUDA calls."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sink_augmented_gqa_b200", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <vector>
#include "sched_slots.cuh"

static long long now = 0;          // a clock of queued work
static bool fail_create = false, fail_wait = false;
struct Ev { long long recorded = -1; };
struct Fake {
  using Status = int;
  using Stream = int;
  using Event = Ev*;
  static constexpr int kOk = 0;
  static long long waited;         // how far back the last wait reached
  static int create(Event* e) { if (fail_create) return 6; *e = new Ev; waited = -1; return 0; }
  static int wait(Stream, Event e) { if (fail_wait) return 6; waited = e->recorded; return 0; }
  static int record(Event e, Stream) { e->recorded = ++now; return 0; }
};
long long Fake::waited = -1;

#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  sa::SchedSlots<Fake> s;
  std::vector<long long> queued(sa::kEagerSchedSlots, -1);   // when a slot's counters were last put to use
  for (int i = 0; i < 300; ++i) {
    const bool fails = i % 7 == 3;
    int got = -1;
    const int r = s.run(i % 2, false, [&](int slot) {
      got = slot;
      if (queued[slot] >= 0 && Fake::waited < queued[slot]) return 99;   // its kernel may still be running
      queued[slot] = ++now;                                             // the kernel is queued ...
      return fails ? 6 : 0;                                             // ... and a launch behind it fails
    });
    CHECK(r == (fails ? 6 : 0));
    CHECK(got == i % sa::kEagerSchedSlots);
  }
  int last = -1;
  for (int i = 0; i < 200; ++i) {   // captured: one slot after the other, failed or not
    const int r = s.run(0, true, [&](int slot) {
      const int want = sa::kEagerSchedSlots + i % sa::kGraphSchedSlots;
      last = slot;
      return slot == want ? (i % 5 == 2 ? 6 : 0) : 99;
    });
    CHECK(r == (i % 5 == 2 ? 6 : 0) && last >= sa::kEagerSchedSlots);
  }
  // a slot that could not be made ready is not launched on, and is the next call's
  const uint64_t at = s.eager_next;
  fail_wait = true;
  bool ran = false;
  CHECK(s.run(0, false, [&](int) { ran = true; return 0; }) == 6 && !ran && s.eager_next == at);
  sa::SchedSlots<Fake> t;
  fail_create = true;
  CHECK(t.run(0, false, [&](int) { ran = true; return 0; }) == 6 && !ran && t.eager_next == 0);
  printf("ok\n");
  return 0;
}
"""


def test_a_failed_launch_uses_its_slot_up(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "slots.cpp", tmp_path / "slots"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-pthread", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout
