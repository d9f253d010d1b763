"""Between two barriers of the tile kernel nothing in LDS is both written and read (no GPU).

attn_order.hpp, which the kernel follows, is compiled for the host with steps that record the
wave's accesses: the number of barriers met so far, and for each buffer the tile whose values the
wave reads or writes there.  A copy counts as a write until the wave waits for it.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "weight_only_quantized_affine_amd", "csrc")
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "attn_order.hpp"
using namespace ql;

// interval kind buffer place tile: a read (R) or write (W) of what belongs to `tile`; P: copies that
// are in flight when a barrier is met
template <int ST> struct Record {
  int interval = 0, base = 0, copies = 0, n = 0;
  bool clean;
  void say(char kind, const char* what, int at, int t) { std::printf("%d %c %s%d %d\n", interval, kind, what, at, base + t); }
  template <class Of> void operator()(Of, int t) {
    switch (Of::value) {
      case AttnStep::kBarrier:
        if (copies) std::printf("%d P copies %d\n", interval, copies);
        ++interval;
        break;
      case AttnStep::kPages: break;
      case AttnStep::kCopyK:
        say('W', "k", attn_stage<ST>(t), t);
        say('W', "seen", attn_seen_at(t), t);
        ++copies;
        break;
      case AttnStep::kCopyV: say('W', "v", attn_stage<ST>(t), t); ++copies; break;
      case AttnStep::kWait: copies = 0; break;
      case AttnStep::kScores: say('R', "k", attn_stage<ST>(t), t); break;
      case AttnStep::kWeights: say('R', "seen", attn_seen_at(t), t); break;
      case AttnStep::kProducts:
        say('R', "v", attn_stage<ST>(t), t);
        if (clean) say('C', "clean", attn_clean_at(t), t);
        if (t + 1 < n) say('R', "k", attn_stage<ST>(t + 1), t + 1);
        break;
      case AttnStep::kIdle: break;
    }
  }
};
template <int ST> void run(bool copier, bool late, bool idle, int n0, int n1) {
  Record<ST> r;
  r.clean = ST > 2;
  for (int n : {n0, n1}) {  // two items, one after the other
    r.n = n;
    attn_tile_order<ST>(n, copier, late, idle, r);
    r.base += 1000;
  }
  std::printf("%d B barriers 0\n", r.interval);
}
int main(int, char** v) {
  const int st = std::atoi(v[1]), copier = std::atoi(v[2]), late = std::atoi(v[3]), idle = std::atoi(v[4]);
  const int n0 = std::atoi(v[5]), n1 = std::atoi(v[6]);
  st == 2 ? run<2>(copier, late, idle, n0, n1) : run<3>(copier, late, idle, n0, n1);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++") or "/opt/rocm/llvm/bin/clang++"
    at = tmp_path_factory.mktemp("order")
    (at / "order.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(at / "order.cpp"), "-o", str(at / "order")], check=True)
    return str(at / "order")


# two stages: four waves, all copying, none late; three: four that copy and four that run behind
WAVES = {2: [(1, 0, 0), (1, 0, 1)], 3: [(1, 0, 0), (1, 0, 1), (0, 1, 0), (0, 1, 1)]}


@pytest.mark.parametrize("stages", [2, 3])
@pytest.mark.parametrize("first,second", [(1, 1), (1, 7), (2, 3), (3, 1), (4, 4), (7, 2), (9, 12)])
def test_no_interval_reads_what_it_writes(program, stages, first, second):
    reads, writes = {}, {}
    for flags in WAVES[stages]:
        wave = ("early", "late")[flags[1]] + (", idle" if flags[2] else "")
        out = subprocess.run([program, *map(str, (stages, *flags, first, second))], check=True, capture_output=True, text=True)
        for line in out.stdout.splitlines():
            interval, kind, what, tile = line.split()
            assert kind != "P", f"{wave}: copies in flight at barrier {interval}"
            if kind in "RC":
                reads.setdefault((int(interval), what), set()).add((wave, int(tile)))
            if kind in "WC":  # (the finite copy: any wave may write it, all of one tile the same values)
                writes.setdefault((int(interval), what), set()).add((wave, int(tile), kind))
    for at, wrote in writes.items():
        same = {t for _, t, k in wrote if k == "C"}
        if same:
            assert len(same) == 1, (at, wrote)
        else:
            assert at not in reads, f"interval {at[0]}: {at[1]} is written by {wrote} and read by {reads[at]}"
            assert len({t for _, t, _ in wrote}) == 1, (at, wrote)
    # what a wave reads was written before, and by nothing newer
    for (interval, what), got in reads.items():
        for wave, tile in got:
            if what.startswith("clean"):
                continue
            before = [(i, t) for (i, w), ws in writes.items() if w == what and i < interval for _, t, _ in ws]
            assert before and max(before)[1] == tile, (interval, what, wave, tile)


def test_all_waves_meet_the_same_barriers(program):
    for stages, kinds in WAVES.items():
        for items in ((1, 1), (2, 5), (7, 3)):
            last = set()
            for flags in kinds:
                out = subprocess.run([program, *map(str, (stages, *flags, *items))], check=True, capture_output=True, text=True)
                last.add(out.stdout.splitlines()[-1])
            assert len(last) == 1, (stages, items, last)
