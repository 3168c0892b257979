"""The cut of a paged decode's batch into runs: the code that the kernels run
(csrc/runs.cuh), compiled for the host and played through on ragged batches."""
import ctypes
import os
import random
import subprocess

import pytest

from gqa_attention_rope_b200 import build as B

PROGRAM = r"""
#include <vector>
#include "runs.cuh"
using namespace la::dpg;
// Plays the runs of a batch and the two joins. 0, or the number of the first thing that is wrong.
extern "C" int play(int B, int Hkv, const int* nst, int max_runs, int* longest, int* shortest) {
  auto stages = [&](int b) { return nst[b]; };
  int total = 0, units = 0;
  std::vector<int> cost_at(B + 1), unit_at(B + 1);
  for (int b = 0; b < B; ++b) {
    cost_at[b] = total, unit_at[b] = units;
    total += cost_of(nst[b]) * Hkv, units += nst[b] * Hkv;
  }
  cost_at[B] = total, unit_at[B] = units;
  if (total == 0) return 0;
  const int n = max_runs < total ? max_runs : total;
  const Cut cut(total, n);
  if (cut.start(0) != 0 || cut.start(n) != total) return 1;
  struct Part { int pair, first, units; };
  std::vector<int> seen(units, 0), whole(B * Hkv, 0);
  std::vector<Part> slot(2 * n, Part{-1, 0, 0});
  std::vector<int> ends(n, -1), ends_first(n, -1);
  *longest = 0, *shortest = 1 << 30;
  int next = 0;
  for (int run = 0; run < n; ++run) {
    const int c0 = cut.start(run), c1 = cut.start(run + 1) - 1;
    if (c1 < c0 || cut.run_of(c0) != run || cut.run_of(c1) != run) return 2;
    if (c1 - c0 + 1 > *longest) *longest = c1 - c0 + 1;
    if (c1 - c0 + 1 < *shortest) *shortest = c1 - c0 + 1;
    int b0 = 0, b1 = 0;
    while (cost_at[b0 + 1] <= c0) ++b0;
    while (cost_at[b1 + 1] <= c1) ++b1;
    const RunBegin begin(c0, cost_at[b0], unit_at[b0], nst[b0]);
    const int u0 = begin.unit, u1 = run_end(c1, cost_at[b1], unit_at[b1], nst[b1]);
    if (u0 != next || u1 < u0) return 3;  // runs meet
    next = u1;
    if (u0 == u1) continue;
    Cursor c{b0, begin.g, begin.s, nst[b0]};
    int seg_first = u0 - c.s;
    for (int u = u0; u < u1; ++u) {
      if (c.b >= B || c.g >= Hkv || c.s >= c.nst || unit_at[c.b] + c.g * c.nst + c.s != u) return 4;
      ++seen[u];
      const bool last = u + 1 == u1;
      if (c.s + 1 == c.nst || last) {  // the segment ends: as the kernel's finish
        const int pair = c.b * Hkv + c.g, seg_end = seg_first + c.nst;
        if (seg_first >= u0 && seg_end <= u1) {
          ++whole[pair];
        } else {
          Part& p = slot[slot_of(run, seg_first >= u0)];
          if (p.pair >= 0) return 5;  // one pair per slot
          const int from = seg_first > u0 ? seg_first : u0, to = seg_end < u1 ? seg_end : u1;
          p = Part{pair, from - seg_first, to - from};
          if (seg_first < u0 && seg_end <= u1) {
            if (ends[run] >= 0) return 6;  // at most one pair that began before ends in a run
            ends[run] = pair;
            ends_first[run] = cut.run_of(begin.first_cost);
          }
        }
        if (!last) {
          Cursor far = c;
          advance(stages, B, Hkv, c, 1);
          advance(stages, B, Hkv, far, 1);
          if (far.b != c.b || far.g != c.g || far.s != c.s) return 7;
          seg_first = u + 1;
        }
      } else {
        ++c.s;
      }
    }
    Cursor jump{b0, begin.g, begin.s, nst[b0]};  // as the loading lanes go, many units at once
    for (int u = u0; u < u1; u += 32, advance(stages, B, Hkv, jump, 32))
      if (unit_at[jump.b] + jump.g * jump.nst + jump.s != u) return 8;
  }
  if (next != units) return 9;
  for (int u = 0; u < units; ++u)
    if (seen[u] != 1) return 10;
  // the joins: by head from the costs, by run from `ends`; each finds all of a pair's rows, in order
  std::vector<int> joined(B * Hkv, 0);
  for (int b = 0; b < B; ++b) {
    for (int g = 0; g < Hkv && nst[b] > 0; ++g) {
      const int pair = b * Hkv + g, at = cost_at[b] + g * cost_of(nst[b]);
      const int r0 = first_run(cut, at), r1 = last_run(cut, at, nst[b]);
      if ((r0 == r1) != (whole[pair] == 1) || whole[pair] > 1) return 11;
      if (r0 == r1) continue;
      int rows = 0;
      for (int r = r0; r <= r1; ++r) {
        const Part& p = slot[slot_of(r, r == r0)];
        if (p.pair != pair || p.first != rows) return 12;
        rows += p.units;
      }
      if (rows != nst[b]) return 13;
      if (ends[r1] != pair || ends_first[r1] != r0) return 14;
      ++joined[pair];
    }
  }
  int in_ends = 0, in_joined = 0;
  for (int x : ends) in_ends += x >= 0;
  for (int x : joined) in_joined += x;
  return in_ends == in_joined ? 0 : 15;
}
"""


@pytest.fixture(scope="module")
def play(tmp_path_factory):
    folder = tmp_path_factory.mktemp("runs")
    src, lib = folder / "play.cpp", folder / "play.so"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I" + os.path.join(B.PKG, "csrc"),
                           str(src), "-o", str(lib)])
    fn = ctypes.CDLL(str(lib)).play

    def call(Hkv, nst, max_runs):
        a, b = ctypes.c_int(), ctypes.c_int()
        st = fn(len(nst), Hkv, (ctypes.c_int * len(nst))(*nst), max_runs, ctypes.byref(a), ctypes.byref(b))
        assert st == 0, (st, Hkv, nst, max_runs)
        return a.value, b.value
    return call


def test_every_unit_once_and_every_partial_result_joined(play):
    rng = random.Random(3)
    for _ in range(3000):
        B = rng.choice([1, 1, 2, 3, 7, 20, 70])
        top = rng.choice([1, 2, 7, 40, 600])
        nst = [0 if rng.random() < 0.2 else rng.randint(1, top) for _ in range(B)]
        play(rng.choice([1, 2, 3, 8]), nst, rng.choice([1, 2, 5, 17, 296, 512]))


def test_the_edges_of_the_cut(play):
    for runs in (1, 2, 6, 7, 8, 296):
        for Hkv in (1, 8):
            for nst in ([1], [0, 1, 0], [2], [1] * 64, [0] * 5, [2048], [1, 2048, 1], [5, 6, 7, 8], [295], [296], [297]):
                play(Hkv, nst, runs)


def test_runs_are_of_equal_cost(play):
    longest, shortest = play(8, [1 + 37 * i % 500 for i in range(64)], 296)
    assert longest - shortest <= 1
