"""What the tile kernel writes into LDS over a cache in 4 bits falls on nothing that is read (no GPU).

As test_host_attention_order.py for a kernel whose copies are loads into registers (and a write of the
bits of the keys to be seen): the products that follow them, or a wait, write V of the next tile and K of
the one behind it, products also where nothing was loaded for them, behind the last tile.
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

// interval kind buffer place tile: a read (R) or write (W) of what belongs to `tile`; X: a copy of what is not
// the tile that the products write, or one that would lose an earlier one; S: places that products write
// whether or not something was loaded for them
template <int ST> struct Record {
  int interval = 0, base = 0, k = -1, v = -1, n = 0;
  bool clean, copier;
  void say(char kind, const char* what, int at, int t) { std::printf("%d %c %s%d %d\n", interval, kind, what, at, base + t); }
  void put() {
    if (v >= 0) say('W', "v", attn_stage<ST>(v), v);
    if (k >= 0) say('W', "k", attn_stage<ST>(k), k);
    v = k = -1;
  }
  void put_products(int tv) {
    if ((v >= 0 && v != tv) || (k >= 0 && k != tv + 1)) say('X', "copy", 0, tv);
    if (v < 0) say('S', "v", attn_stage<ST>(tv), tv);
    if (k < 0) say('S', "k", attn_stage<ST>(tv + 1), tv + 1);
    put();
  }
  template <class Of> void operator()(Of, int t) {
    switch (Of::value) {
      case AttnStep::kBarrier: ++interval; break;
      case AttnStep::kPages: break;
      case AttnStep::kCopyK:
        if (k >= 0 && k != 0) say('X', "lost", 0, t);  // K of an item's first tile is written before the next is loaded
        if (k == 0) say('W', "k", attn_stage<ST>(k), k);
        say('W', "seen", attn_seen_at(t), t);
        k = t;
        break;
      case AttnStep::kCopyV:
        if (v >= 0) say('X', "lost", 0, t);
        v = t;
        break;
      case AttnStep::kWait: put(); break;
      case AttnStep::kScores:
        say('R', "k", attn_stage<ST>(t), t);
        break;
      case AttnStep::kWeights: say('R', "seen", attn_seen_at(t), t); break;
      case AttnStep::kProducts:
        say('R', "v", attn_stage<ST>(t), t);
        if (clean) say('C', "clean", attn_clean_at(t), t);
        if (t + 1 < n) say('R', "k", attn_stage<ST>(t + 1), t + 1);
        if (copier) put_products(t + 1);
        break;
      case AttnStep::kIdle: break;
    }
  }
};
template <int ST> void run(bool copier, bool late, bool idle, int n0, int n1) {
  Record<ST> r;
  r.clean = ST > 2;
  r.copier = copier;
  for (int n : {n0, n1}) {  // two items, one after the other
    r.n = n;
    attn_tile_order<ST>(n, copier, late, idle, r);
    if (r.k >= 0 || r.v >= 0) r.say('X', "left", 0, 0);
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
    at = tmp_path_factory.mktemp("order4")
    (at / "order.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(at / "order.cpp"), "-o", str(at / "order")], check=True)
    return str(at / "order")


# two stages: four waves, all copying, none late; three: four that copy and four that run behind
WAVES = {2: [(1, 0, 0), (1, 0, 1)], 3: [(1, 0, 0), (1, 0, 1), (0, 1, 0), (0, 1, 1)]}


def lines(program, stages, flags, items):
    out = subprocess.run([program, *map(str, (stages, *flags, *items))], check=True, capture_output=True, text=True)
    return [line.split() for line in out.stdout.splitlines()]


@pytest.mark.parametrize("stages", [2, 3])
@pytest.mark.parametrize("items", [(1, 1), (1, 7), (2, 3), (3, 1), (4, 4), (7, 2), (9, 12)])
def test_no_interval_reads_what_it_writes(program, stages, items):
    reads, writes, spare = {}, {}, {}
    for flags in WAVES[stages]:
        wave = ("early", "late")[flags[1]] + (", idle" if flags[2] else "")
        for interval, kind, what, tile in lines(program, stages, flags, items):
            at = (int(interval), what)
            assert kind != "X", f"{wave}: {what} at tile {tile}"
            if kind in "RC":
                reads.setdefault(at, set()).add((wave, int(tile)))
            if kind in "WC":
                writes.setdefault(at, set()).add((wave, int(tile), kind))
            if kind == "S":
                spare.setdefault(at, set()).add((wave, int(tile)))
    for at, wrote in writes.items():
        same = {t for _, t, k in wrote if k == "C"}
        if same:  # the finite copy: any wave may write it, all of one tile the same values
            assert len(same) == 1, (at, wrote)
        else:
            assert at not in reads, f"interval {at[0]}: {at[1]} is written by {wrote} and read by {reads[at]}"
            assert len({t for _, t, _ in wrote}) == 1, (at, wrote)
    for at, wrote in spare.items():  # what no copy loaded falls on nothing that is read or written
        assert at not in reads and at not in writes, (at, wrote, reads.get(at), writes.get(at))
    # what a wave reads was written by every copying wave before, and nothing newer or spare came after
    for (interval, what), got in reads.items():
        for wave, tile in got:
            if what.startswith("clean"):
                continue
            before = [(i, t) for (i, w), ws in writes.items() if w == what and i < interval for _, t, _ in ws]
            assert before and max(before)[1] == tile, (interval, what, wave, tile)
            kinds = {k for (i, w), ws in writes.items() if w == what and i < interval for k, t, _ in ws if t == tile}
            assert len(kinds) == sum(copier for copier, _, _ in WAVES[stages]), (interval, what, tile, kinds)
            last = max(before)[0]
            assert not any(w == what and last <= i < interval for i, w in spare), (interval, what, tile)
